// Routed expert projection of a few tokens on 4-bit weights with a scale per
// group along K (rom_expert_proj_w4), and the quantiser that writes them
// (rom_quant_expert_weights_w4).
//
//   w[e][n][c] = (q[e][n][c] - 8) * s[e][n][c / group],  q in 0 .. 15
//   out[slot]  = r_slot * sum_c x[token][c] w[e_slot][:, c]
//
// What bounds it: the bytes of the selected experts' weights (half a byte per
// weight, a quarter of bf16), so only experts that some token selected are
// read, once for up to 32 of their tokens. The matrix instruction is the
// warp-level m16n8k16, not tcgen05: its A operand (16 weight rows) comes from
// registers, so a code goes from the loaded word to the tensor core without a
// pass through shared memory, which for 2 bytes per weight would cost as much
// time as reading the 4-bit weights from HBM. The codes are integers -8 .. 7,
// exact in bf16; products with bf16 activations are exact in float32, sums are
// float32, and a group's sum is multiplied by its scale in float32.
//
// Storage, a 1 KB tile per 16 rows x 128 columns, [E][N/16][K/128] tiles (N and
// K rounded up; codes 8 and scales 0 there): byte h*512 + (g*4 + t)*16 + b holds
// what lane g*4 + t loads for row g + 8h; as four 32-bit words, nibble p of word
// i is the column 32 i + 16 ((p >> 1) & 1) + 4 t + 2 (p & 1) + (p >> 2). So a
// 16-byte load per lane and row half brings the A operands of 8 steps of 16
// columns, nibbles p and p + 4 lie in one register's two halves after a shift
// and a mask, and the B operand of a step is 8 contiguous bytes of the token's
// row. A warp's loads are whole contiguous kilobytes.
#include <cuda_bf16.h>

#include <algorithm>

#include "rom_internal.cuh"
#include "sm100_ptx.cuh"

namespace rom {
namespace {

constexpr int kW4Warps = 8;                  // 16 weight rows each
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kW4Rows = kW4Warps * 16;       // weight rows per CTA
constexpr int kW4Stage = 2;                  // 128-column blocks per ring stage
constexpr int kW4Cols = kW4Stage * 128;
// Bytes of a token's row in a stage: 256 columns and a pad that puts the rows
// of a quad column 32 bytes apart modulo 128 (conflict-free 8-byte reads).
constexpr int kW4RowBytes = kW4Cols * 2 + 32;
constexpr int kW4ScaleBytes = 128;           // per warp and block: 16 rows, up to 4 groups
constexpr int kW4WarpBytes = kW4Stage * (1024 + kW4ScaleBytes);
constexpr int kW4RedPitch = kW4Rows + 4;
constexpr int kW4MaxTokens = 64;

struct W4Params {
  const __nv_bfloat16* x;
  const uint8_t* q[2];
  const __nv_bfloat16* s[2];
  const int32_t* topk_idx;
  const float* topk_w;  // null: unweighted
  void* out;
  int T, K, N, E, k;
  int nt, kb;           // 16-row tiles, 128-column blocks
  int splits;           // CTAs of a cluster that share a row block's columns
  int max_active;       // upper bound of the experts in use
  int to_token;         // bf16 rows in token order (k == 1), else float32 slot rows
  int* status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(full ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// Two codes of a word (bits SH .. SH + 3 and SH + 16 .. SH + 19) as bf16 q - 8:
// the bits of 128 + q (q < 16 sits in the mantissa's last 4 bits), less 136.
template <int SH>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  const uint32_t v = ((w >> SH) & 0x000f000fu) | 0x43004300u;
  const uint32_t c = 0x43084308u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

struct W4Ctl {
  uint32_t mask[2];  // experts in use
  int count;
  int slot[kW4MaxTokens * kMaxTopK];  // this expert's slots, in order
};

template <int NB, int STAGES>
constexpr size_t w4_smem_bytes() {
  const size_t ring = static_cast<size_t>(STAGES) * (kW4Warps * kW4WarpBytes + NB * 8 * kW4RowBytes);
  const size_t red = static_cast<size_t>(NB) * 8 * kW4RedPitch * 4;
  return (ring > red ? ring : red) + sizeof(W4Ctl);
}

// One CTA: 128 weight rows of one expert (and of one of up to two matrices)
// times the expert's tokens, over its part of the columns. NB: 8-token blocks
// held at a time; an expert with more tokens is passed over again. GS: steps of
// 16 columns that share a scale (group / 16).
template <int NB, int STAGES, int GS>
__global__ void __launch_bounds__(kW4Threads, 2) w4_proj_kernel(const W4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kTok = NB * 8;
  constexpr int kStageBytes = kW4Warps * kW4WarpBytes + kTok * kW4RowBytes;
  constexpr size_t kCtlAt = w4_smem_bytes<NB, STAGES>() - sizeof(W4Ctl);
  W4Ctl& ctl = *reinterpret_cast<W4Ctl*>(smem + kCtlAt);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int row_blk = blockIdx.x / p.splits;
  const int mat = blockIdx.y / p.max_active;
  const int nth = blockIdx.y - mat * p.max_active;
  const int nslots = p.T * p.k;

  if (tid < 2) ctl.mask[tid] = 0;
  pdl_wait();  // the router's outputs and x are complete from here
  __syncthreads();
  for (int i = tid; i < nslots; i += kW4Threads) {
    const int e = p.topk_idx[i];
    if (e >= 0 && e < p.E)
      atomicOr(&ctl.mask[e >> 5], 1u << (e & 31));
    else if (p.status)
      atomicExch(p.status, kStatusRouting);
  }
  __syncthreads();
  // the nth expert in use; every CTA of a cluster leaves or stays together
  const uint64_t mask = ctl.mask[0] | (static_cast<uint64_t>(ctl.mask[1]) << 32);
  if (nth >= __popcll(mask)) return;
  uint64_t rest = mask;
  for (int i = 0; i < nth; ++i) rest &= rest - 1;
  const int e = __ffsll(static_cast<long long>(rest)) - 1;
  if (warp == 0) {
    int n = 0;
    for (int i = 0; i < nslots; i += 32) {
      const bool mine = i + lane < nslots && p.topk_idx[i + lane] == e;
      const unsigned b = __ballot_sync(0xffffffffu, mine);
      if (mine) ctl.slot[n + __popc(b & ((1u << lane) - 1u))] = i + lane;
      n += __popc(b);
    }
    if (lane == 0) ctl.count = n;
  }
  __syncthreads();
  const int count = ctl.count;

  const int tile = row_blk * kW4Warps + warp;
  const bool has_tile = tile < p.nt;
  const int64_t tile0 = (static_cast<int64_t>(e) * p.nt + (has_tile ? tile : 0)) * p.kb;
  const uint8_t* qw = (mat ? p.q[1] : p.q[0]) + tile0 * 1024 + lane * 16;
  constexpr int kGroups = 8 / GS;                 // scales per row and block
  constexpr int kScaleLanes = 2 * kGroups;        // 16-byte pieces of a block's scales
  const uint8_t* sw =
      reinterpret_cast<const uint8_t*>(mat ? p.s[1] : p.s[0]) + tile0 * (kScaleLanes * 16) + lane * 16;
  // this CTA's blocks of 128 columns
  const int b0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / p.splits);
  const int b1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / p.splits);
  const int iters = (b1 - b0 + kW4Stage - 1) / kW4Stage;
  const uint32_t smem0 = smem_u32(smem);

  for (int p0 = 0; p0 < count; p0 += kTok) {
    const int n_tok = min(kTok, count - p0);
    const int n_blk = (n_tok + 7) / 8;
    float acc[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nb][j] = 0.f;

    auto issue = [&](int it) {
      if (it < iters) {
        const uint32_t st = smem0 + (it % STAGES) * kStageBytes;
        const uint32_t ws = st + warp * kW4WarpBytes;
#pragma unroll
        for (int b = 0; b < kW4Stage; ++b) {
          const int kb = b0 + it * kW4Stage + b;
          if (has_tile && kb < b1) {
            const uint8_t* src = qw + static_cast<int64_t>(kb) * 1024;
            cp_async16(ws + b * 1024 + lane * 16, src, true);
            cp_async16(ws + b * 1024 + 512 + lane * 16, src + 512, true);
            if (lane < kScaleLanes)
              cp_async16(ws + kW4Stage * 1024 + b * kW4ScaleBytes + lane * 16,
                         sw + static_cast<int64_t>(kb) * (kScaleLanes * 16), true);
          }
        }
        const uint32_t xs = st + kW4Warps * kW4WarpBytes;
        const int c0 = (b0 + it * kW4Stage) * 128;
        const int cend = min(p.K, b1 * 128);
        for (int i = tid; i < n_blk * 8 * (kW4Cols / 8); i += kW4Threads) {
          const int r = i / (kW4Cols / 8), c = (i % (kW4Cols / 8)) * 8;
          const bool in = r < n_tok && c0 + c < cend;
          const int64_t tok = in ? ctl.slot[p0 + r] / p.k : 0;
          cp_async16(xs + r * kW4RowBytes + c * 2, p.x + tok * p.K + (in ? c0 + c : 0), in);
        }
      }
      cp_async_commit();
    };

#pragma unroll
    for (int it = 0; it < STAGES - 1; ++it) issue(it);
    for (int it = 0; it < iters; ++it) {
      cp_async_wait<STAGES - 2>();
      __syncthreads();
      issue(it + STAGES - 1);
      const uint8_t* st = smem + (it % STAGES) * kStageBytes;
      const uint8_t* ws = st + warp * kW4WarpBytes;
      const uint8_t* xs = st + kW4Warps * kW4WarpBytes + g * kW4RowBytes + t * 8;
#pragma unroll
      for (int b = 0; b < kW4Stage; ++b) {
        if (!has_tile || b0 + it * kW4Stage + b >= b1) continue;  // warp-uniform
        const uint4 qa = *reinterpret_cast<const uint4*>(ws + b * 1024 + lane * 16);
        const uint4 qb = *reinterpret_cast<const uint4*>(ws + b * 1024 + 512 + lane * 16);
        const uint32_t wa[4] = {qa.x, qa.y, qa.z, qa.w}, wb[4] = {qb.x, qb.y, qb.z, qb.w};
        uint32_t a[8][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[2 * i][0] = codes<0>(wa[i]);
          a[2 * i][1] = codes<0>(wb[i]);
          a[2 * i][2] = codes<4>(wa[i]);
          a[2 * i][3] = codes<4>(wb[i]);
          a[2 * i + 1][0] = codes<8>(wa[i]);
          a[2 * i + 1][1] = codes<8>(wb[i]);
          a[2 * i + 1][2] = codes<12>(wa[i]);
          a[2 * i + 1][3] = codes<12>(wb[i]);
        }
        const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(
            ws + kW4Stage * 1024 + b * kW4ScaleBytes);
        float s_lo[kGroups], s_hi[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          s_lo[i] = __bfloat162float(sc[g * kGroups + i]);
          s_hi[i] = __bfloat162float(sc[(g + 8) * kGroups + i]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (nb < n_blk) {  // CTA-uniform
            const uint8_t* xb = xs + nb * 8 * kW4RowBytes + b * 256;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < GS; ++j)
                mma_16816(d, a[i * GS + j],
                          *reinterpret_cast<const uint2*>(xb + (i * GS + j) * 32));
              acc[nb][0] = fmaf(s_lo[i], d[0], acc[nb][0]);
              acc[nb][1] = fmaf(s_lo[i], d[1], acc[nb][1]);
              acc[nb][2] = fmaf(s_hi[i], d[2], acc[nb][2]);
              acc[nb][3] = fmaf(s_hi[i], d[3], acc[nb][3]);
            }
          }
        }
      }
    }

    // The sums meet in shared memory as [token][row] (over the ring, which no
    // copy still writes), are added over the cluster in rank order and stored
    // row-contiguous.
    cp_async_wait<0>();
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (nb < n_blk) {
        float* r0 = red + (nb * 8 + 2 * t) * kW4RedPitch + warp * 16 + g;
        r0[0] = acc[nb][0];
        r0[kW4RedPitch] = acc[nb][1];
        r0[8] = acc[nb][2];
        r0[kW4RedPitch + 8] = acc[nb][3];
      }
    }
    if (p.splits > 1)
      cluster_sync_all();
    else
      __syncthreads();
    const int rows = kW4Rows / p.splits;  // this rank's share of the rows
    for (int i = tid; i < n_tok * rows; i += kW4Threads) {
      const int j = i / rows, r = rank * rows + (i - j * rows);
      const int n = row_blk * kW4Rows + r;
      if (n < p.N) {
        float v = 0.f;
        if (p.splits > 1) {
          const uint32_t at = smem_u32(red + j * kW4RedPitch + r);
          for (int c = 0; c < p.splits; ++c) v += ld_cluster_f32(mapa_shared(at, c));
        } else {
          v = red[j * kW4RedPitch + r];
        }
        const int slot = ctl.slot[p0 + j];
        if (p.topk_w) v *= p.topk_w[slot];
        if (p.to_token)
          static_cast<__nv_bfloat16*>(p.out)[static_cast<int64_t>(slot) * p.N + n] =
              __float2bfloat16_rn(v);
        else
          static_cast<float*>(p.out)[(static_cast<int64_t>(mat) * nslots + slot) * p.N + n] = v;
      }
    }
    // no CTA reuses or leaves its shared memory while another reads it
    __syncwarp();
    if (p.splits > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }
}

template <int NB, int STAGES, int GS>
cudaError_t launch_w4(const W4Params& p, int mats, cudaStream_t stream) {
  auto kern = w4_proj_kernel<NB, STAGES, GS>;
  constexpr size_t smem = w4_smem_bytes<NB, STAGES>();
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int row_blks = (p.nt + kW4Warps - 1) / kW4Warps;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(row_blks * p.splits),
                     static_cast<unsigned>(p.max_active * mats), 1);
  cfg.blockDim = dim3(kW4Threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NB, int STAGES>
cudaError_t launch_w4_group(const W4Params& p, int mats, int group, cudaStream_t stream) {
  switch (group) {
    case 32:
      return launch_w4<NB, STAGES, 2>(p, mats, stream);
    case 64:
      return launch_w4<NB, STAGES, 4>(p, mats, stream);
    default:
      return launch_w4<NB, STAGES, 8>(p, mats, stream);
  }
}

__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xffff0000u);
  v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}

// One warp per 16 x 128 tile; lane (g, t) makes its own 32 codes of the rows g
// and g + 8, so it stores the 16 bytes that the projection's lane loads. The
// scale is rounded to bf16 first and the codes are taken against the rounded
// scale, so its rounding adds no error of its own: s = bf16(max |w| / 7),
// q = 8 + round(w / s) clamped to 0 .. 15 (a group of zeros: s = 0, q = 8).
template <typename WT>
__global__ void __launch_bounds__(256)
    quant_w4_kernel(const WT* __restrict__ w, int64_t tiles, int N, int K, int nt, int kb, int gs,
                    uint8_t* __restrict__ q, __nv_bfloat16* __restrict__ s) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t tile = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (tile >= tiles) return;
  const int b = static_cast<int>(tile % kb);
  const int64_t et = tile / kb;
  const int64_t e = et / nt;
  const int rt = static_cast<int>(et - e * nt);
  const int groups = 8 / gs;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = rt * 16 + h * 8 + g;
    float v[8][4];
    uint32_t m[8];  // per step: bits of the largest |w|
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = b * 128 + j * 16 + t * 4;
      v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.f;
      if (n < N && c < K) load4(w + (e * N + n) * K + c, v[j]);
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m[j] = max(m[j], __float_as_uint(v[j][i]) & 0x7fffffffu);
      m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 1));
      m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 2));
    }
    // over the group's steps: pairs, fours or all eight
#pragma unroll
    for (int j = 0; j < 8; j += 2) m[j] = m[j + 1] = max(m[j], m[j + 1]);
    if (gs >= 4)
#pragma unroll
      for (int j = 0; j < 8; j += 4) m[j] = m[j + 1] = m[j + 2] = m[j + 3] = max(m[j], m[j + 2]);
    if (gs >= 8) {
      const uint32_t all = max(m[0], m[4]);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = all;
    }
    uint32_t words[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // a group that holds an infinity or a NaN has a NaN scale
      const bool finite = m[j] < 0x7f800000u;
      const __nv_bfloat16 sb = __float2bfloat16_rn(
          finite ? __fdiv_rn(__uint_as_float(m[j]), 7.0f) : __uint_as_float(0x7fffffffu));
      const float sf = __bfloat162float(sb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int code = 8;
        if (finite && sf > 0.f)
          code = 8 + static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(v[j][i], sf)), -8.f), 7.f));
        words[j >> 1] |= static_cast<uint32_t>(code) << (4 * ((j & 1) * 2 + (i >> 1) + (i & 1) * 4));
      }
      if (t == 0 && j % gs == 0) s[(tile * 16 + h * 8 + g) * groups + j / gs] = sb;
    }
    *reinterpret_cast<uint4*>(q + tile * 1024 + h * 512 + lane * 16) =
        make_uint4(words[0], words[1], words[2], words[3]);
  }
}

}  // namespace

cudaError_t launch_w4_proj(const void* x, int T, int K, const void* q0, const void* s0,
                           const void* q1, const void* s1, int N, int E, int k, int group,
                           const int32_t* topk_idx, const float* topk_w, void* out, bool to_token,
                           int* status, cudaStream_t stream) {
  W4Params p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.q[0] = static_cast<const uint8_t*>(q0);
  p.q[1] = static_cast<const uint8_t*>(q1);
  p.s[0] = static_cast<const __nv_bfloat16*>(s0);
  p.s[1] = static_cast<const __nv_bfloat16*>(s1);
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  p.out = out;
  p.T = T;
  p.K = K;
  p.N = N;
  p.E = E;
  p.k = k;
  p.nt = (N + 15) / 16;
  p.kb = (K + 127) / 128;
  p.to_token = to_token ? 1 : 0;
  p.status = status;
  p.max_active = std::min(E, T * k);
  const int mats = q1 ? 2 : 1;
  // Few row blocks (few tokens or a small N): the CTAs of a cluster share a
  // row block's columns, until there are about two CTAs per SM or a CTA is
  // left with fewer than 4 blocks of 128 columns.
  const int64_t units = static_cast<int64_t>((p.nt + kW4Warps - 1) / kW4Warps) * p.max_active * mats;
  p.splits = 1;
  while (p.splits < 8 && units * p.splits < 2 * static_cast<int64_t>(device_sm_count()) &&
         p.kb / (p.splits * 2) >= 4)
    p.splits *= 2;
  if (T <= 8) return launch_w4_group<1, 4>(p, mats, group, stream);
  if (T <= 16) return launch_w4_group<2, 4>(p, mats, group, stream);
  return launch_w4_group<4, 3>(p, mats, group, stream);
}

cudaError_t launch_quant_w4(const void* w, bool bf16, int E, int N, int K, int group, void* q,
                            void* s, cudaStream_t stream) {
  const int nt = (N + 15) / 16, kb = (K + 127) / 128;
  const int64_t tiles = static_cast<int64_t>(E) * nt * kb;
  const unsigned grid = static_cast<unsigned>((tiles + 7) / 8);
  if (bf16)
    quant_w4_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(w), tiles, N, K, nt,
                                              kb, group / 16, static_cast<uint8_t*>(q),
                                              static_cast<__nv_bfloat16*>(s));
  else
    quant_w4_kernel<<<grid, 256, 0, stream>>>(static_cast<const float*>(w), tiles, N, K, nt, kb,
                                              group / 16, static_cast<uint8_t*>(q),
                                              static_cast<__nv_bfloat16*>(s));
  return cudaGetLastError();
}

}  // namespace rom
