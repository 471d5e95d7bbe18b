// Routed expert projection of a few tokens on 4-bit weights with a scale per
// group along K (rom_expert_proj_w4), and the quantiser that writes them
// (rom_quant_expert_weights_w4).
//
//   w[e][n][c] = (q[e][n][c] - 8) * s[e][n][c / group],  q in 0 .. 15
//   out[slot]  = r_slot * sum_c x[token][c] w[e_slot][:, c]
//
// What bounds it: the bytes of the selected experts' weights (half a byte per
// weight, a quarter of bf16) for few tokens, the instructions and shared-memory
// reads of the products for many. Only experts that some token selected are
// read, once for up to 24 of their tokens. The matrix instruction is the
// warp-level m16n8k16: its A operand (16 weight rows) comes from registers, so a
// code goes from the loaded word to the tensor core without a pass through
// shared memory. One form on tcgen05 was measured, and slower: with the weights in
// TMEM as A (M = 128) an MMA of 16 or 32 tokens takes 60 cycles to issue, 8 per 128 x
// 128 block, and every unit of 128 rows waits for its accumulators (63 us for 64
// tokens over 4 experts of 10240 x 4096, this kernel 34 to 36). Weights unpacked into
// shared memory for it were not tried. The codes are integers
// -8 .. 7, exact in bf16; products with bf16 activations are exact in float32,
// sums are float32, and a group's sum is multiplied by its scale in float32.
//
// Storage, a 1 KB tile per 16 rows x 128 columns, [E][N/16][K/128] tiles (N and
// K rounded up; codes 8 and scales 0 there): byte h*512 + (g*4 + t)*16 + b holds
// what lane g*4 + t loads for row g + 8h; as four 32-bit words, nibble p of word
// i is the column 32 i + 16 ((p >> 1) & 1) + 4 t + 2 (p & 1) + (p >> 2). So a
// 16-byte load per lane and row half brings the A operands of 8 steps of 16
// columns, nibbles p and p + 4 lie in one register's two halves after a shift
// and a mask, and the B operand of a step is 8 contiguous bytes of the token's
// row. A warp's loads are whole contiguous kilobytes.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "rom_internal.cuh"
#include "sm100_ptx.cuh"

namespace rom {
namespace {

constexpr int kW4MaxWarps = 9;               // consumer warps of a CTA, 16 weight rows each
constexpr int kW4MinWarps = 4;
constexpr int kW4Stage = 2;                  // 128-column blocks per ring stage
constexpr int kW4Cols = kW4Stage * 128;
// Bytes of a token's row in a stage: its columns and a pad that puts the rows
// 32 bytes apart modulo 128 (conflict-free 8-byte reads of the B operand).
constexpr int kW4RowBytes = kW4Cols * 2 + 32;
constexpr int kW4WarpBytes = kW4Stage * (1024 + 128);  // a warp's codes and scales
constexpr int kW4MaxTokens = 64;
constexpr int kW4MaxSlots = kW4MaxTokens * kMaxTopK;
constexpr int kW4MaxStages = 6;
constexpr int kW4MostSmem = 110 * 1024;   // of each of two CTAs on an SM
constexpr int kW4ThirdSmem = 73 * 1024;   // of each of three
// CTAs that an SM holds: their registers set it. Of one token block, three with up to
// 7 consumer warps at 80 a thread, or with up to 9 at 64 (kTight); of more, two of 9
// at 96. The kernels are bounded to these, so that it is so with any compiler.
__host__ __device__ constexpr int w4_resident(int nb) { return nb == 1 ? 3 : 2; }
__host__ __device__ constexpr int w4_registers(int nb, bool tight) {
  return tight ? 64 : nb == 1 ? 80 : 96;
}
// (with the producer warp)
constexpr bool w4_fits(int nb, int warps, bool tight) {
  return w4_resident(nb) * (warps + 1) * 32 * w4_registers(nb, tight) <= 65536;
}
static_assert(w4_fits(1, 7, false) && w4_fits(1, kW4MaxWarps, true) && w4_fits(2, kW4MaxWarps, false) &&
                  w4_fits(3, kW4MaxWarps, false),
              "an SM's registers hold the CTAs that the shape of the work counts on");

struct W4Params {
  const __nv_bfloat16* x;
  const int32_t* topk_idx;
  const float* topk_w;  // null: unweighted
  void* out;
  int T, K, N, E, k;
  int nt, kb;           // 16-row tiles, 128-column blocks
  int splits;           // CTAs of a cluster that share a row block's columns
  int max_active;       // upper bound of the experts in use
  int resident;         // CTAs that an SM is to hold
  int passes;           // CTAs that share an expert's passes over its tokens
  int stages;           // of the ring
  int to_token;         // bf16 rows in token order (k == 1), else float32 slot rows
  int* status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(full ? 16 : 0)
               : "memory");
}
// One arrival on *bar (counted in its phase) once this thread's cp.async so far
// have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// d += a b^T, and d = a b^T (16 x 8 x 16).
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.f));
}

// Two codes of a word (bits SH .. SH + 3 and SH + 16 .. SH + 19) as bf16 q - 8, by the
// well-known conversion of small integers through a power of two's mantissa (widely
// published for 4-bit weights in this form): the bf16 numbers 128 .. 255 are 128 + m
// with m the 7 bits behind the point, so a code's bits put there make 128 + q, and
// taking 136 away is exact. One three-input logic instruction and one packed
// multiply-add, both spelled out: left to the compiler the two logic steps stay two
// (64 tokens on 4 experts of 10240 x 4096: 37.3 us, 34.3 so), and it turns a
// multiplication by one into a subtraction, which takes 36.1.
template <int SH>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  constexpr int kAndOr = (0xf0 & 0xcc) | 0xaa;  // the truth table of (a & b) | c
  constexpr uint32_t kCodes = 0x000f000f, k128 = 0x43004300;       // bf16 128 twice
  constexpr uint32_t kOne = 0x3f803f80, kMinus136 = 0xc308c308;    // bf16 1 and -136
  uint32_t v, d;
  asm("lop3.b32 %0, %1, %2, %3, %4;" : "=r"(v) : "r"(w >> SH), "r"(kCodes), "r"(k128), "n"(kAndOr));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(kOne), "r"(kMinus136));
  return d;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

struct W4Ctl {
  uint64_t full[kW4MaxStages], empty[kW4MaxStages];
  uint32_t mask[2];  // experts in use
  int abort;
  int group_count[kW4MaxSlots / 32];  // of this expert's slots, per 32 slots
  int16_t slot[kW4MaxSlots];          // this expert's slots, in order,
  uint8_t tok[kW4MaxSlots];           // their tokens
  float weight[kW4MaxSlots];          // and their routing weights (or 1)
};

// Ring, then the control block.
template <int NB>
__host__ __device__ constexpr int w4_stage_bytes(int warps) {
  return warps * kW4WarpBytes + NB * 8 * kW4RowBytes;
}

// One 16 x 128 tile times NBL blocks of 8 tokens: acc += scale * (codes * x),
// two steps of 16 columns at a time (one word of each row's codes), the chains
// of the token blocks side by side. xs: this lane's first bytes of the first
// block's x.
template <int NBL, int GS, int NB>
__device__ __forceinline__ void w4_tile(const uint4 qa, const uint4 qb, const __nv_bfloat16* sc,
                                        int g, const uint8_t* xs, float (&acc)[NB][4]) {
  constexpr int kGroups = 8 / GS;
  const uint32_t wa[4] = {qa.x, qa.y, qa.z, qa.w}, wb[4] = {qb.x, qb.y, qb.z, qb.w};
  float d[NBL][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a0[4] = {codes<0>(wa[i]), codes<0>(wb[i]), codes<4>(wa[i]), codes<4>(wb[i])};
    const uint32_t a1[4] = {codes<8>(wa[i]), codes<8>(wb[i]), codes<12>(wa[i]), codes<12>(wb[i])};
#pragma unroll
    for (int nb = 0; nb < NBL; ++nb) {
      const uint8_t* xb = xs + nb * 8 * kW4RowBytes + i * 64;
      if (2 * i % GS == 0)
        mma_16816_first(d[nb], a0, *reinterpret_cast<const uint2*>(xb));
      else
        mma_16816(d[nb], a0, *reinterpret_cast<const uint2*>(xb));
    }
#pragma unroll
    for (int nb = 0; nb < NBL; ++nb)
      mma_16816(d[nb], a1,
                *reinterpret_cast<const uint2*>(xs + nb * 8 * kW4RowBytes + i * 64 + 32));
    if ((2 * i + 2) % GS == 0) {
      const int gr = (2 * i) / GS;
      const float lo = __bfloat162float(sc[g * kGroups + gr]);
      const float hi = __bfloat162float(sc[(g + 8) * kGroups + gr]);
#pragma unroll
      for (int nb = 0; nb < NBL; ++nb) {
        acc[nb][0] = fmaf(lo, d[nb][0], acc[nb][0]);
        acc[nb][1] = fmaf(lo, d[nb][1], acc[nb][1]);
        acc[nb][2] = fmaf(hi, d[nb][2], acc[nb][2]);
        acc[nb][3] = fmaf(hi, d[nb][3], acc[nb][3]);
      }
    }
  }
}

// Tensor maps of the codes (1 KB tiles) and scales of up to two matrices.
struct W4Maps {
  CUtensorMap q[2], s[2];
};

// One CTA: 16 weight rows per consumer warp of one expert (and of one of up to
// two matrices) times the expert's tokens, over its part of the columns. The
// last warp feeds the ring, so the consumers spend no instruction on addresses:
// the codes and the scales of all warps' tiles come in one TMA copy each (a
// bulk copy per tile and row cost 90 cycles apiece to issue, 3600 a stage), the
// tokens' rows by 16-byte copies that arrive on the stage's barrier. NB: 8-token
// blocks held at a time; an expert with more tokens is passed over again. GS:
// steps of 16 columns that share a scale (group / 16). Every wait is bounded.
//
// kTight: 64 registers, for three CTAs of 8 or 9 consumer warps on an SM where
// there are as many (19 tokens, top-2 of 16 experts of 2004 x 1000, Conv+Gate: 12.9
// us; 14.7 with three of 7; both called in a loop, the weights in L2). Elsewhere the
// bound costs more than it gives (one token, 8 experts of 4096 x 2048, top-2: 7.2 us,
// 6.7 without).
template <int NB, int GS, bool kTight>
__global__ void __maxnreg__(w4_registers(NB, kTight))
    w4_proj_kernel(const __grid_constant__ W4Maps maps, const W4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kTok = NB * 8;
  const int warps = (blockDim.x >> 5) - 1;  // consumers
  const int stage_bytes = w4_stage_bytes<NB>(warps);
  W4Ctl& ctl = *reinterpret_cast<W4Ctl*>(smem + p.stages * stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int row_blk = blockIdx.x / p.splits;
  const int mat = blockIdx.y / p.max_active;
  const int nth = blockIdx.y - mat * p.max_active;
  const int nslots = p.T * p.k;

  if (tid < 2) ctl.mask[tid] = 0;
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&ctl.full[i], 1 + 32);  // the TMA copies, the producer's lanes
      mbar_init(&ctl.empty[i], warps);
    }
    ctl.abort = 0;
    fence_barrier_init();
  }
  pdl_wait();  // the router's outputs and x are complete from here
  __syncthreads();
  // Every thread keeps its slots' experts; the slots of 32 consecutive threads
  // are one group.
  constexpr int kMine = (kW4MaxSlots + (kW4MinWarps + 1) * 32 - 1) / ((kW4MinWarps + 1) * 32);
  int my_e[kMine];
  float my_w[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int sl = i * blockDim.x + tid;
    my_e[i] = -1;
    if (sl < nslots) {
      const int v = p.topk_idx[sl];
      my_w[i] = p.topk_w ? p.topk_w[sl] : 1.f;
      if (v >= 0 && v < p.E) {
        my_e[i] = v;
        atomicOr(&ctl.mask[v >> 5], 1u << (v & 31));
      } else if (p.status) {
        atomicExch(p.status, kStatusRouting);
      }
    }
  }
  __syncthreads();
  // the nth expert in use; every CTA of a cluster leaves or stays together
  const uint64_t mask = ctl.mask[0] | (static_cast<uint64_t>(ctl.mask[1]) << 32);
  if (nth >= __popcll(mask)) return;
  uint64_t rest = mask;
  for (int i = 0; i < nth; ++i) rest &= rest - 1;
  const int e = __ffsll(static_cast<long long>(rest)) - 1;
  const int groups = (nslots + 31) / 32;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int grp = i * (warps + 1) + warp;
    if (grp < groups) {
      const unsigned b = __ballot_sync(0xffffffffu, my_e[i] == e);
      if (lane == 0) ctl.group_count[grp] = __popc(b);
    }
  }
  __syncthreads();
  int count = 0;
  for (int grp = 0; grp < groups; ++grp) {
    const int n = ctl.group_count[grp];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (grp == i * (warps + 1) + warp) {  // warp-uniform
        const unsigned b = __ballot_sync(0xffffffffu, my_e[i] == e);
        if (my_e[i] == e) {
          const int at = count + __popc(b & ((1u << lane) - 1u)), sl = grp * 32 + lane;
          ctl.slot[at] = static_cast<int16_t>(sl);
          ctl.tok[at] = static_cast<uint8_t>(sl / p.k);
          ctl.weight[at] = my_w[i];
        }
      }
    }
    count += n;
  }
  const int first = blockIdx.z * kTok;
  if (first >= count) return;  // cluster-uniform
  __syncthreads();
  volatile int* abort_flag = &ctl.abort;

  constexpr int kScaleBytes = 32 * (8 / GS);  // of a 16 x 128 tile
  // this CTA's blocks of 128 columns
  const int b0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / p.splits);
  const int b1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / p.splits);
  const int tiles = min(warps, p.nt - row_blk * warps);  // warps with rows
  int stage = 0;
  uint32_t phase = 0;

  for (int p0 = first; p0 < count; p0 += gridDim.z * kTok) {
    const int n_tok = min(kTok, count - p0);
    const int n_blk = (n_tok + 7) / 8;
    float acc[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nb][j] = 0.f;

    if (warp == warps) {
      // ------------------------------------------------ producer
      // (a last row block's missing tiles: the next expert's, or zeros, not used)
      const int tile0 = e * p.nt + row_blk * warps;
      const CUtensorMap* mq = &maps.q[mat];
      const CUtensorMap* ms = &maps.s[mat];
      uint32_t src[kTok];  // 16-byte pieces; lane l: columns 8 l .. + 7 of a stage
#pragma unroll
      for (int r = 0; r < kTok; ++r)
        src[r] = (r < n_tok ? ctl.tok[p0 + r] : 0u) * (static_cast<uint32_t>(p.K) / 8u) + lane;
      const uint4* xsrc = reinterpret_cast<const uint4*>(p.x);
      uint32_t issued = 0, last_par = 0;
      for (int kb = b0; kb < b1; kb += kW4Stage) {
        if (!mbar_wait_warp(&ctl.empty[stage], phase ^ 1u, abort_flag, p.status)) break;
        uint8_t* st = smem + stage * stage_bytes;
        if (lane == 0) {
          mbar_arrive_expect_tx(&ctl.full[stage], warps * kW4Stage * (1024 + kScaleBytes));
          tma_load_3d(st, mq, &ctl.full[stage], 0, kb, tile0);
          tma_load_3d(st + warps * kW4Stage * 1024, ms, &ctl.full[stage], 0, kb, tile0);
        }
        const uint32_t xd = smem_u32(st + warps * kW4WarpBytes + lane * 16);
        const int c = kb * 128 + lane * 8;
        const bool in = c < min(p.K, b1 * 128);  // other columns: zeros
#pragma unroll
        for (int r = 0; r < kTok; ++r)
          if (r < n_tok) cp_async16(xd + r * kW4RowBytes, xsrc + (in ? src[r] + kb * 16 : 0u), in);
        cp_async_arrive(&ctl.full[stage]);
        issued |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | (phase << stage);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // every copy has landed before the ring is used for the sums
      int never = 0;
      for (int i = 0; i < p.stages; ++i)
        if ((issued >> i) & 1u) mbar_wait(&ctl.full[i], (last_par >> i) & 1u, &never, p.status);
    } else {
      // ------------------------------------------------ consumers
      for (int kb = b0; kb < b1; kb += kW4Stage) {
        if (!mbar_wait_warp(&ctl.full[stage], phase, abort_flag, p.status)) break;
        const uint8_t* st = smem + stage * stage_bytes;
        const uint8_t* ws = st + warp * (kW4Stage * 1024);
        const uint8_t* ss = st + warps * (kW4Stage * 1024) + warp * (kW4Stage * kScaleBytes);
        const uint8_t* xs = st + warps * kW4WarpBytes + g * kW4RowBytes + t * 8;
        if (warp < tiles) {
#pragma unroll
          for (int b = 0; b < kW4Stage; ++b) {
            if (b > 0 && kb + b >= b1) break;
            const uint4 qa = *reinterpret_cast<const uint4*>(ws + b * 1024 + lane * 16);
            const uint4 qb = *reinterpret_cast<const uint4*>(ws + b * 1024 + 512 + lane * 16);
            const __nv_bfloat16* sc =
                reinterpret_cast<const __nv_bfloat16*>(ss + b * kScaleBytes);
            if (NB == 1 || n_blk == 1)
              w4_tile<1, GS>(qa, qb, sc, g, xs + b * 256, acc);
            else if (NB == 2 || n_blk == 2)
              w4_tile<NB < 2 ? 1 : 2, GS>(qa, qb, sc, g, xs + b * 256, acc);
            else
              w4_tile<NB < 3 ? 1 : 3, GS>(qa, qb, sc, g, xs + b * 256, acc);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.empty[stage]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }

    // The sums meet in shared memory as [token][row] (over the ring, whose
    // copies have all landed and been read), are added over the cluster in rank
    // order and stored row-contiguous.
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
    const int pitch = warps * 16 + 4;
    if (warp < warps) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (nb < n_blk) {
          float* r0 = red + (nb * 8 + 2 * t) * pitch + warp * 16 + g;
          r0[0] = acc[nb][0];
          r0[pitch] = acc[nb][1];
          r0[8] = acc[nb][2];
          r0[pitch + 8] = acc[nb][3];
        }
      }
    }
    fence_async_shared();  // before the next pass's copies into the same bytes
    __syncwarp();
    if (p.splits > 1)
      cluster_sync_all();
    else
      __syncthreads();
    const int rows = warps * 16 / p.splits;  // this rank's share of the rows
    const int row0 = rank * rows, n0 = row_blk * warps * 16 + row0;
    const int n_rows = *abort_flag ? 0 : min(rows, p.N - n0);
    // a warp per token, or several that share its rows
    const int share = max(1, (warps + 1) / n_tok), turn = (warps + 1) / share;
    for (int j = warp / share; j < n_tok; j += turn) {
      const float r = ctl.weight[p0 + j];
      const int slot = ctl.slot[p0 + j];
      const float* from = red + j * pitch + row0;
      __nv_bfloat16* o16 = static_cast<__nv_bfloat16*>(p.out) + static_cast<int64_t>(slot) * p.N + n0;
      float* o32 =
          static_cast<float*>(p.out) + (static_cast<int64_t>(mat) * nslots + slot) * p.N + n0;
#pragma unroll 4
      for (int i = warp % share * 32 + lane; i < n_rows; i += 32 * share) {
        float v;
        if (p.splits > 1) {
          const uint32_t at = smem_u32(from + i);
          v = 0.f;
          for (int c = 0; c < p.splits; ++c) v += ld_cluster_f32(mapa_shared(at, c));
        } else {
          v = from[i];
        }
        v *= r;
        if (p.to_token)
          o16[i] = __float2bfloat16_rn(v);
        else
          o32[i] = v;
      }
    }
    // no CTA reuses or leaves its shared memory while another reads it
    __syncwarp();
    if (p.splits > 1)
      cluster_sync_all();
    else
      __syncthreads();
    if (*abort_flag && p.splits == 1) return;
  }
}

template <int NB, int GS, bool kTight = false>
cudaError_t launch_w4(W4Params p, const W4Maps& maps, int warps, int mats, cudaStream_t stream) {
  if constexpr (NB == 1 && !kTight)
    if (p.resident > 2 && warps > 7) return launch_w4<NB, GS, true>(p, maps, warps, mats, stream);
  auto kern = w4_proj_kernel<NB, GS, kTight>;
  // Once per device: the most shared memory a launch asks for, and the largest
  // carve-out, so that several CTAs fit an SM.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !((ready.load() >> dev) & 1u)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4MostSmem);
    if (err != cudaSuccess) return err;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (err != cudaSuccess) return err;
    if (dev < 64) ready.fetch_or(uint64_t(1) << dev);
  }
  const int row_blks = (p.nt + warps - 1) / warps;
  const int stage = w4_stage_bytes<NB>(warps);
  const int budget = (p.resident > 2 ? kW4ThirdSmem : kW4MostSmem) -
                     static_cast<int>(sizeof(W4Ctl));
  p.stages = std::min(kW4MaxStages, budget / stage);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(row_blks * p.splits),
                     static_cast<unsigned>(p.max_active * mats),
                     static_cast<unsigned>(p.passes));
  cfg.blockDim = dim3(static_cast<unsigned>((warps + 1) * 32), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.stages) * stage + sizeof(W4Ctl);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

template <int NB>
cudaError_t launch_w4_group(const W4Params& p, const W4Maps& maps, int warps, int mats, int group,
                            cudaStream_t stream) {
  switch (group) {
    case 32:
      return launch_w4<NB, 2>(p, maps, warps, mats, stream);
    case 64:
      return launch_w4<NB, 4>(p, maps, warps, mats, stream);
    default:
      return launch_w4<NB, 8>(p, maps, warps, mats, stream);
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
  // Token blocks of 8 held at a time: enough for an expert with two standard
  // deviations more tokens than an even routing gives it (one with more is
  // passed over again, its weights then coming from L2): fewer blocks leave room
  // for more CTAs. 19 tokens, top-2 of 16 experts: 13.0 us with 1, 18.1 with 3; 32
  // tokens, top-1 of 4: 29.0 with 2, 43 with 1.
  const double even = static_cast<double>(T) * k / E;
  const double most = std::min(static_cast<double>(T), even + 2.0 * std::sqrt(even));
  const int nb = most <= 8.0 ? 1 : most <= 16.0 ? 2 : 3;
  // Shape of the work: CTAs of `warps` 16-row tiles, `splits` of them (a
  // cluster) sharing the columns of one row block, `passes` sharing an expert's
  // token blocks where it has more than nb. The cost is an SM's: the CTAs that
  // come to it times what one goes through, its warps' 16 x 128 tiles, dearer
  // where few warps are resident, and the cluster's hand-over of its sums, in
  // tiles (fewer where a tile takes longer for its tokens). The constants are the
  // best of a grid over 75 shapes timed in every form, 3 % above the best form on
  // average, geometrically; each shape in a loop on one set of weights, most of which
  // fit L2. Measured so, us, at 4 experts of 10240 x 4096: one token 10.7 (9 warps, 2
  // splits; 12.6 with 4 and 1, 14.0 with 9 and 4), 64 tokens 36.3 (9 and 1; 44 with 5,
  // 47 with 8; later changes brought the 36.3 to 34.3); 4 experts of 154 x 3960, 30 tokens,
  // top-3: 9.3 (4 and 8; 14.2 with 4 and 2). With every call's weights from HBM the
  // chosen forms take 11.8, 35.8 and 12.2; the others were not timed so.
  const double used = std::ceil(E * (1.0 - std::pow(1.0 - static_cast<double>(k) / E, T)) - 0.1);
  const double blocks = std::max(1.0, static_cast<double>(T) * k / used / 8.0);
  const double hand_over = 96.0 / std::sqrt(blocks);
  const int passes = std::max(1, static_cast<int>(std::ceil(blocks / nb - 0.1)));
  const int sms = device_sm_count();
  int warps = kW4MaxWarps;
  double best = 1e30;
  for (int z = 1; z <= passes; z = z < passes ? passes : passes + 1) {
    for (int s = 1; s <= 8 && s <= p.kb; s *= 2) {
      for (int w = kW4MaxWarps; w >= kW4MinWarps; --w) {
        const double ctas = std::ceil(((p.nt + w - 1) / w) * used * mats * s * z / sms);
        const double resident = std::min(ctas, static_cast<double>(w4_resident(nb))) * w;
        const double tiles = w * ((p.kb + s - 1) / s) * (1.0 + 11.0 / resident);
        const double cost = ctas * passes / z * (tiles + (s > 1 ? hand_over : 0.0));
        if (cost < best * 0.999) {
          best = cost;
          warps = w;
          p.splits = s;
          p.passes = z;
          p.resident = static_cast<int>(std::min<double>(ctas, w4_resident(nb)));
        }
      }
    }
  }
  W4Maps maps;
  const int64_t tiles = static_cast<int64_t>(E) * p.nt;
  for (int i = 0; i < mats; ++i)
    if (!make_tile_map(&maps.q[i], i ? q1 : q0, 1024, p.kb, tiles, kW4Stage, warps) ||
        !make_tile_map(&maps.s[i], i ? s1 : s0, 32 * (128 / group), p.kb, tiles, kW4Stage, warps))
      return cudaErrorInvalidValue;
  if (mats == 1) {
    maps.q[1] = maps.q[0];
    maps.s[1] = maps.s[0];
  }
  if (nb == 1) return launch_w4_group<1>(p, maps, warps, mats, group, stream);
  if (nb == 2) return launch_w4_group<2>(p, maps, warps, mats, group, stream);
  return launch_w4_group<3>(p, maps, warps, mats, group, stream);
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
