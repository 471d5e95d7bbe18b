// Grouped bf16 GEMM of the RoM expert projections on the 5th-generation tensor
// cores (tcgen05.mma, fp32 accumulators in TMEM, operands staged by TMA).
// ("Routing Mamba ..." chapterpal summary page, Knowl 1: H_t, G_t and O_t are
// linear projections by the selected experts; Swimba project page, Extended
// abstract: routed in-projection experts.)
//
// For expert e the rows offsets[e] .. offsets[e+1]-1 of A ([R][K] bf16,
// expert-contiguous) are multiplied by B_e^T, B_e = W[e] stored [N][K]. The
// expert row counts are read on the device: each CTA rebuilds the tile list
// from `offsets` (no host synchronisation). Tiles never straddle experts;
// rows past an expert's end are computed and discarded at the store.
//
// Tile: 256 rows x 256 accumulator columns x 64-element K steps, computed
// by a pair of CTAs on two SMs (a 2-CTA cluster, tcgen05.mma.cta_group::2):
// each CTA holds 128 of the rows and half of the 256 B columns in its shared
// memory and receives its rows' 128 x 256 fp32 accumulator in its own TMEM.
//   Conv+Gate: the 256 columns are 128 columns of W_in (held by CTA 0) next
//   to the same 128 columns of W_g (CTA 1), so one MMA of N = 256 yields u
//   and z side by side, and the epilogue forms h = u * SiLU(z) (top-1) or
//   stores u and z per slot (top-k).
//   Out / in-projection: 256 output columns, scaled by r in the epilogue (a
//   last tile of 128 columns when N % 256 == 128: the weight rows past N are
//   zero-filled by TMA and those columns are not stored).
// CTA: persistent (one pair of CTAs per pair of SMs), 6 warps (10 in 8 bits):
//   warp 0  TMA producer (one thread), 6- or 7-stage ring (32 KB/stage/CTA)
//   warp 1  TMEM allocator; in CTA 0 also the MMA issuer (one thread)
//   warps 2-5  epilogue; warp w reads TMEM lanes 32*(w%4) .. +31 (in 8 bits,
//              where a tile's MMAs take half the time, warps 2-9: two per lane group)
// Two TMEM accumulators (2 x 256 columns) let the epilogue of one tile run
// while the MMAs of the next tile proceed. Every wait is bounded.
// Few routed rows (decode) take a swap-AB kernel instead (below).
//
// The same kernels run the products in 8 bits (rom_expert_proj_q8, kQ8): rows
// and weights in e4m3 with a float32 scale per row and per output feature,
//   value[p][n] = ((sum_c a8[p][c] w8[e][n][c]) * sa[p]) * sw[e][n].
// A 128-byte row of a stage then holds 128 elements of K instead of 64 and one
// MMA takes 32 of them instead of 16, so tiles, ring, descriptors and barriers
// are those of bf16 and a stage of the same bytes does twice the work. The
// scales are constant along K: they multiply the float32 accumulator in the
// epilogue, before SiLU and before the routing weight.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "rom_internal.cuh"
#include "sm100_ptx.cuh"

namespace rom {
namespace {

constexpr int BM = 128;
constexpr int BKB = 128;  // bytes of K per stage and row: one swizzle row
constexpr int BK = BKB / 2;
template <bool kQ8>
constexpr int kBK = kQ8 ? BKB : BKB / 2;  // elements of K per stage
constexpr int UMMA_N = 256;
constexpr uint32_t TMEM_COLS = 2 * UMMA_N;
constexpr int kThreads = 192;
// Out / in-projection calls with at most this many routed rows use the
// swap-AB kernel (weights on the MMA's M side).
constexpr int64_t kSwapMaxRows = 1024;
// In 8 bits, calls with at most this many routed rows per expert on average, as
// measured on even routings (us, swap-AB against the pair kernel, K 2048, N 2048
// unless stated): 8 rows per expert of 8, K 4096: 12.7 / 18.4; 32 of 64, N 1024: 36 /
// 66; 64 of 8: 14.9 / 15.1; 91 of 33, K and N 1024: 22.0 / 19.5; 128 of 8: 19.8 / 15.7.
// Conv+Gate at N 4096: 8 of 8: 25.2 / 31.3; 32 of 8: 27.7 / 32.4; 64 of 8: 34.3 / 33.3;
// 128 of 8: 43.6 / 34.2. The rows of each expert are on the device, so the rule goes by
// the mean; where the rows sit on a few experts the pair kernel would be the faster
// one, up to twice (64 experts, N 1024, weights from HBM; Out, then Conv+Gate). 64 rows
// per expert, even: 33.9 / 38.0, 39.9 / 59.1; on half of them: 26.3 / 20.2, 36.4 / 30.3;
// all on one: 25.7 / 13.0, 36.1 / 18.3. 32 per expert, even: 31.0 / 36.7, 37.9 / 58.2; on
// half: 16.2 / 18.6, 22.4 / 28.4; on one: 15.7 / 11.4, 21.9 / 12.6. 96 per expert, even:
// 46.7 / 39.1, 64.9 / 59.9; on one: 35.1 / 17.0, 49.7 / 23.9.
constexpr int64_t kSwapMaxRowsPerExpertQ8 = 64;

struct Params {
  const int32_t* offsets;
  const int32_t* sorted_slot;
  const float* topk_w;
  void* out;
  int64_t R;
  int K;
  int N;
  int E;
  int k;
  int n_tiles_n;
  int* status;
  // the dense small-batch in-projection: every token's experts (else null)
  const int32_t* topk_idx;
  // dense small-batch kernel: weights in the tile-major layout
  // [E][N/128][K/64][128][64] (one 16 KB block per weight tile)
  int w_tiled;
  // 8-bit products: scales of the sorted rows [R] and of the output features
  // [E][N] (of W_in and W_g, or of the one matrix)
  const float* a_scale;
  const float* w0_scale;
  const float* w1_scale;
};

// 8-bit products: acc[j] = (acc[j] * sa) * sw[j] for 32 columns, the scales of the
// columns read from shared memory as 8 uniform 16-byte loads. One scale after the
// other, in every kernel: their product alone may leave float32's range or its
// normal numbers where the value does not.
template <bool kQ8>
__device__ __forceinline__ void apply_scales(uint32_t (&acc)[32], float sa, const float* sw) {
  if (kQ8) {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const float4 s = reinterpret_cast<const float4*>(sw)[v];
      acc[4 * v + 0] = __float_as_uint(__uint_as_float(acc[4 * v + 0]) * sa * s.x);
      acc[4 * v + 1] = __float_as_uint(__uint_as_float(acc[4 * v + 1]) * sa * s.y);
      acc[4 * v + 2] = __float_as_uint(__uint_as_float(acc[4 * v + 2]) * sa * s.z);
      acc[4 * v + 3] = __float_as_uint(__uint_as_float(acc[4 * v + 3]) * sa * s.w);
    }
  }
}

// u * SiLU(z) = u * z / (1 + e^-z), with the fast exp and divide intrinsics:
// their relative error (~1e-6) is far below the bf16 rounding of h (2^-9),
// and for z < -88 (e^-z = inf) the quotient is 0 as SiLU's limit.
__device__ __forceinline__ float silu_gate(float u, float z) {
  return u * __fdividef(z, 1.0f + __expf(-z));
}

// Slot of sorted row `prow` (row order itself for a dense projection, which
// passes no sorted_slot) and the expert row bounds (one expert owning all R
// rows when no offsets are passed).
__device__ __forceinline__ int64_t slot_of(const Params& p, int64_t prow) {
  return p.sorted_slot ? static_cast<int64_t>(p.sorted_slot[prow]) : prow;
}
__device__ __forceinline__ int offset_of(const Params& p, int i) {
  return p.offsets ? p.offsets[i] : (i == 0 ? 0 : static_cast<int>(p.R));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Epilogue of one accumulator tile for one warp: thread i reads TMEM lane
// t_row.lane + i, i.e. sorted row `prow` (stored only when `valid`), the
// 32-column chunks c0 .. c1 - 1 of output columns n0 .. n0 + w - 1 (w = 128 for
// the gate modes, whose z columns follow the w u columns in TMEM, 256 otherwise;
// half of that for the half tiles of a last wave). The float32 outputs (per-slot
// partials), and in 8 bits the bf16 rows too, go through the warp's staging tile
// `stg`, so that a store instruction writes consecutive bytes of a few rows; the
// bf16 rows of bf16 products, half as wide and half as frequent, are stored
// directly in 16-byte pieces, which measured faster for them. `own` and, for the
// columns' scales, 512 bytes at `sws` are the 8-bit epilogue's: it is handed the
// tile's slots, weights and scales, which the caller read during the tile before
// (9272 rows of K 464 and N 2944 over 16 experts: 38.6 us with these loads, the
// rows' addresses and an arrival that waited for the stores in each chunk's way,
// 27.2 so).
// What a tile's row needs besides its accumulator: its slot, routing weight (or
// 1) and scale, and of a lane the scales of up to 128 columns (four of its own:
// of the chunks' columns, and of W_g's behind W_in's for the gate modes).
struct EpiRow {
  int64_t slot = 0;
  float r = 0.f, sa = 0.f, sw[4] = {0.f, 0.f, 0.f, 0.f};
};
template <int MODE, bool kQ8>
__device__ __forceinline__ EpiRow epilogue_row(const Params& p, bool valid, int64_t prow, int e,
                                               int n0, int c0, int c1) {
  EpiRow o;
  if (valid) {
    if (MODE != kEpiGateH) o.slot = slot_of(p, prow);
    if (kQ8) o.sa = p.a_scale[prow];
    // no routing weights passed: r = 1
    if (MODE == kEpiScaleToken || MODE == kEpiScaleSlots) o.r = p.topk_w ? p.topk_w[o.slot] : 1.f;
  }
  if (kQ8) {
    constexpr bool kGate = (MODE == kEpiGateH || MODE == kEpiGateSlots);
    const int64_t at = static_cast<int64_t>(e) * p.N;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + (kGate ? i & 1 : i), n = n0 + c * 32 + (threadIdx.x & 31);
      if (c < c1 && n < p.N) o.sw[i] = (kGate && i > 1 ? p.w1_scale : p.w0_scale)[at + n];
    }
  }
  return o;
}

template <int MODE, bool kQ8>
__device__ __forceinline__ void epilogue_rows(const Params& p, uint32_t t_row, bool valid,
                                              int64_t prow, const EpiRow& own, int n0, int w,
                                              int c0, int c1, float* stg, float* sws) {
  const float sa = own.sa;
  // the output rows that this lane stores from the staging tile
  constexpr bool kF32 = (MODE == kEpiGateSlots || MODE == kEpiScaleSlots);
  int rows[8];
  if (kF32 || kQ8) {
    const int64_t row = MODE == kEpiGateH        ? prow
                        : MODE == kEpiScaleToken ? own.slot / p.k
                                                 : own.slot;
    const int mine = valid ? static_cast<int>(row) : -1, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      rows[i] = __shfl_sync(0xffffffffu, mine,
                            kF32 ? 4 * i + (lane >> 3) : (8 * i + (lane >> 2)) & 31);
  }
  if (kQ8) {  // the columns' scales, 32 of a chunk in a row
#pragma unroll
    for (int i = 0; i < 4; ++i) sws[i * 32 + (threadIdx.x & 31)] = own.sw[i];
    __syncwarp();
  }
  if (MODE == kEpiGateH) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      uint32_t u[32], z[32];
      tmem_ld32(t_row + c * 32, u);
      tmem_ld32(t_row + w + c * 32, z);
      tmem_ld_wait();
      apply_scales<kQ8>(u, sa, sws + (c - c0) * 32);
      apply_scales<kQ8>(z, sa, sws + (c - c0) * 32 + 64);
      if (valid || kQ8) {
        uint4* dst = reinterpret_cast<uint4*>(out + prow * p.N + n0 + c * 32);
        uint4 ws[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint4 w;
          w.x = pack_bf16(silu_gate(__uint_as_float(u[8 * v + 0]), __uint_as_float(z[8 * v + 0])),
                          silu_gate(__uint_as_float(u[8 * v + 1]), __uint_as_float(z[8 * v + 1])));
          w.y = pack_bf16(silu_gate(__uint_as_float(u[8 * v + 2]), __uint_as_float(z[8 * v + 2])),
                          silu_gate(__uint_as_float(u[8 * v + 3]), __uint_as_float(z[8 * v + 3])));
          w.z = pack_bf16(silu_gate(__uint_as_float(u[8 * v + 4]), __uint_as_float(z[8 * v + 4])),
                          silu_gate(__uint_as_float(u[8 * v + 5]), __uint_as_float(z[8 * v + 5])));
          w.w = pack_bf16(silu_gate(__uint_as_float(u[8 * v + 6]), __uint_as_float(z[8 * v + 6])),
                          silu_gate(__uint_as_float(u[8 * v + 7]), __uint_as_float(z[8 * v + 7])));
          if (kQ8)
            ws[v] = w;
          else
            dst[v] = w;
        }
        if (kQ8)
          store_tile_bf16(reinterpret_cast<uint8_t*>(stg), ws, rows, out + n0 + c * 32, p.N);
      }
    }
  } else if (MODE == kEpiGateSlots) {
    float* out = static_cast<float*>(p.out);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      uint32_t u[32], z[32];
      tmem_ld32(t_row + c * 32, u);
      tmem_ld32(t_row + w + c * 32, z);
      tmem_ld_wait();
      apply_scales<kQ8>(u, sa, sws + (c - c0) * 32);
      apply_scales<kQ8>(z, sa, sws + (c - c0) * 32 + 64);
      float f[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(u[j]);
      store_tile_f32(stg, f, rows, out + n0 + c * 32, p.N);
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(z[j]);
      store_tile_f32(stg, f, rows, out + p.R * p.N + n0 + c * 32, p.N);
    }
  } else {
    const int64_t slot = own.slot;
    const float r = own.r;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      if (n0 + c * 32 >= p.N) break;  // partial last tile (N % 256 == 128)
      uint32_t a[32];
      tmem_ld32(t_row + c * 32, a);
      tmem_ld_wait();
      apply_scales<kQ8>(a, sa, sws + (c - c0) * 32);
      if (MODE == kEpiScaleToken) {
        if (valid || kQ8) {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
          uint4* dst = reinterpret_cast<uint4*>(out + (slot / p.k) * p.N + n0 + c * 32);
          uint4 ws[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 w;
            w.x = pack_bf16(r * __uint_as_float(a[8 * v + 0]), r * __uint_as_float(a[8 * v + 1]));
            w.y = pack_bf16(r * __uint_as_float(a[8 * v + 2]), r * __uint_as_float(a[8 * v + 3]));
            w.z = pack_bf16(r * __uint_as_float(a[8 * v + 4]), r * __uint_as_float(a[8 * v + 5]));
            w.w = pack_bf16(r * __uint_as_float(a[8 * v + 6]), r * __uint_as_float(a[8 * v + 7]));
            if (kQ8)
              ws[v] = w;
            else
              dst[v] = w;
          }
          if (kQ8)
            store_tile_bf16(reinterpret_cast<uint8_t*>(stg), ws, rows, out + n0 + c * 32, p.N);
        }
      } else {
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = r * __uint_as_float(a[j]);
        float* out = static_cast<float*>(p.out);
        store_tile_f32(stg, f, rows, out + n0 + c * 32, p.N);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// SM-pair variant (cluster of two CTAs, tcgen05.mma.cta_group::2): a pair
// tile is 256 rows x 256 accumulator columns. CTA v of the pair loads rows
// 128v .. 128v+127 of the tile's A rows and half of the B rows (Conv+Gate:
// CTA 0 the 128 W_in columns, CTA 1 the same 128 W_g columns; Out: CTA v
// the output columns 128v .. 128v+127), so each SM streams 32 KB per K step
// instead of 48 KB, and the 128 x 256 accumulator of its own rows lands in
// its own TMEM, where its own epilogue warps read it, one row per
// thread. Protocol:
//   full[s]   lives in CTA 0: CTA 0's producer arms it with both CTAs'
//             bytes; both producers' TMA loads complete on it.
//   empty[s]  one per CTA: the MMA commit arrives on both (multicast).
//   tfull[a]  one per CTA: the commit after a tile's last MMA, multicast.
//   tempty[a] lives in CTA 0: the epilogue warps of each CTA arrive
//             (CTA 1's through the cluster window).
// A CTA never exits while the other may still touch its shared memory or
// TMEM: both end at a cluster barrier that every path reaches after bounded
// waits.
constexpr int PM = 256;                      // rows per pair tile
// Ring depth: 7 stages for the bf16-output modes, 6 (plus the epilogue warps'
// staging tiles) for the float32-output modes.
constexpr int P_MAX_STAGES = 7;
// 8-bit products, whose tiles' MMAs take half of bf16's time, have 8 epilogue
// warps (two per 32 rows, half of the columns each) and stage their bf16 outputs
// too; their staging tiles cost a stage.
template <int MODE, bool kQ8>
struct PairGeo {
  static constexpr bool kF32 = (MODE == kEpiGateSlots || MODE == kEpiScaleSlots);
  static constexpr int kEpiWarps = kQ8 ? 8 : 4;
  static constexpr int kStages = (kF32 ? 6 : 7) - (kQ8 ? 1 : 0);
  static constexpr int kStageTile =  // bytes per epilogue warp
      kF32 ? kStageFloats * 4 : kQ8 ? kStageBf16Bytes : 0;
  // bytes of its columns' scales, behind it
  static constexpr int kScales = kQ8 ? 512 : 0;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
};
constexpr int P_A_BYTES = BM * BK * 2;       // 16 KB: this CTA's 128 rows
constexpr int P_B_BYTES = 128 * BK * 2;      // 16 KB: this CTA's half of B
constexpr int P_STAGE_BYTES = P_A_BYTES + P_B_BYTES;

struct PairCtl {
  uint64_t full[P_MAX_STAGES];
  uint64_t empty[P_MAX_STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int tile_start[kMaxExperts + 1];
  int off[kMaxExperts + 1];
  int mt[kMaxExperts];
};

constexpr size_t kPairCtlBytes = (sizeof(PairCtl) + 15) / 16 * 16;
// ring, control block, the epilogue warps' staging tiles, alignment slack
template <int MODE, bool kQ8>
constexpr size_t pair_smem_bytes() {
  using Geo = PairGeo<MODE, kQ8>;
  return Geo::kStages * P_STAGE_BYTES + kPairCtlBytes +
         Geo::kEpiWarps * (Geo::kStageTile + Geo::kScales) + 1024;
}

template <int MODE, bool kQ8>
__global__ void __launch_bounds__(PairGeo<MODE, kQ8>::kThreads, 1)
    tc_pair_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB0,
                        const __grid_constant__ CUtensorMap tmB1,
                        const __grid_constant__ CUtensorMap tmB0h,
                        const __grid_constant__ CUtensorMap tmB1h, const Params p) {
  constexpr bool kGate = (MODE == kEpiGateH || MODE == kEpiGateSlots);
  constexpr int kTileN = kGate ? 128 : 256;  // output columns per tile
  constexpr int P_STAGES = PairGeo<MODE, kQ8>::kStages;
  constexpr int kEpiWarps = PairGeo<MODE, kQ8>::kEpiWarps;
  extern __shared__ uint8_t smem_raw[];
  // Same 1024-byte aligned offset in both CTAs (same kernel, same static
  // layout), as the pair MMA reads the peer's operands at the leader's offsets.
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  PairCtl& ctl = *reinterpret_cast<PairCtl*>(smem + P_STAGES * P_STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  const uint32_t rank = cluster_ctarank();
  const bool leader = (rank == 0);
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int npairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < P_STAGES; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&ctl.tfull[a], 1);
      mbar_init(&ctl.tempty[a], 2 * kEpiWarps);
    }
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(kGate && !leader ? &tmB1 : &tmB0);
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctl.tmem_base, TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (kQ8) pdl_wait();  // the sorted rows and their routing are complete from here
  for (int i = threadIdx.x; i <= E; i += PairGeo<MODE, kQ8>::kThreads)
    ctl.off[i] = offset_of(p, i);
  __syncthreads();
  if (threadIdx.x == 0) {
    int run = 0;
    for (int e = 0; e < E; ++e) {
      const int mt = (ctl.off[e + 1] - ctl.off[e] + PM - 1) / PM;
      ctl.mt[e] = mt;
      ctl.tile_start[e] = run;
      run += mt * p.n_tiles_n;
    }
    ctl.tile_start[E] = run;
  }
  tc_fence_before();
  cluster_sync_all();  // barriers initialised in both CTAs before any remote use
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem_base;
  const int total = ctl.tile_start[E];
  const int KB = (p.K + kBK<kQ8> - 1) / kBK<kQ8>;
  volatile int* abort_flag = &ctl.abort;

  auto coords = [&](int tile, int& e, int& m_blk, int& n_blk) {
    e = 0;
    while (tile >= ctl.tile_start[e + 1]) ++e;
    const int local = tile - ctl.tile_start[e];
    n_blk = local / ctl.mt[e];
    m_blk = local - n_blk * ctl.mt[e];
  };
  // Work items of this pair: its whole tiles pair, pair + npairs, ... of the
  // full waves, then its item of the last wave. When the last wave holds at
  // most npairs / 2 tiles, each of them is cut into two halves of N / 2
  // columns (pair 2i and 2i + 1 take tile i's halves), so that wave keeps
  // every pair busy for half a tile's time instead of some pairs for a
  // whole one. half: -1 for a whole tile, else 0 or 1.
  const int full_waves = total / npairs;
  const int rem = total - full_waves * npairs;
  const bool halve = rem > 0 && 2 * rem <= npairs;
  auto item = [&](int j, int& tile, int& half) -> bool {
    if (j < full_waves) {
      tile = pair + j * npairs;
      half = -1;
      return true;
    }
    if (j > full_waves) return false;
    if (halve) {
      if (pair >= 2 * rem) return false;
      tile = full_waves * npairs + pair / 2;
      half = pair & 1;
      return true;
    }
    if (pair >= rem) return false;
    tile = full_waves * npairs + pair;
    half = -1;
    return true;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ TMA producer (both CTAs)
      const CUtensorMap* tmB = (kGate && !leader) ? &tmB1 : &tmB0;
      const CUtensorMap* tmBh = (kGate && !leader) ? &tmB1h : &tmB0h;
      const uint32_t full0 = mapa_shared(smem_u32(&ctl.full[0]), 0);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, last_par = 0;
      bool ok = true;
      int tile, half;
      for (int j = 0; ok && item(j, tile, half); ++j) {
        int e, m_blk, n_blk;
        coords(tile, e, m_blk, n_blk);
        const int row0 = ctl.off[e] + m_blk * PM + static_cast<int>(rank) * BM;
        // B rows of this CTA: whole tile 128 (Conv+Gate: the tile's 128 W_in
        // or W_g rows; Out: its half of the 256 columns), half tile 64
        const int r = static_cast<int>(rank);
        const int brow0 = half < 0 ? (kGate ? n_blk * 128 : n_blk * 256 + r * 128)
                                   : (kGate ? n_blk * 128 + half * 64
                                            : n_blk * 256 + half * 128 + r * 64);
        const CUtensorMap* mb = half < 0 ? tmB : tmBh;
        const uint32_t bytes =
            half < 0 ? 2u * P_STAGE_BYTES : 2u * (P_A_BYTES + P_B_BYTES / 2);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * P_STAGE_BYTES;
          const uint32_t fb = full0 + static_cast<uint32_t>(stage * sizeof(uint64_t));
          if (leader) mbar_arrive_expect_tx(&ctl.full[stage], bytes);
          tma_load_2d_pair(sa, &tmA, fb, kb * kBK<kQ8>, row0);
          tma_load_3d_pair(sa + P_A_BYTES, mb, fb, kb * kBK<kQ8>, brow0, e);
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == P_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (leader) {
        // Every load of both CTAs has landed before the pair can exit.
        int never = 0;
        for (int s = 0; s < P_STAGES; ++s)
          if ((issued >> s) & 1u) mbar_wait(&ctl.full[s], (last_par >> s) & 1u, &never, p.status);
      } else if (!ok) {
        // Aborted: this CTA's loads complete on the leader's barriers, which
        // it cannot wait on; give copies in flight a fixed time to land.
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------ MMA issuer (CTA 0)
      const uint32_t idesc_whole = kQ8 ? idesc_e4m3_f32(PM, UMMA_N) : idesc_bf16_f32(PM, UMMA_N);
      const uint32_t idesc_half =
          kQ8 ? idesc_e4m3_f32(PM, UMMA_N / 2) : idesc_bf16_f32(PM, UMMA_N / 2);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      int tile, half;
      for (int j = 0; ok && item(j, tile, half); ++j) {
        const uint32_t idesc = half < 0 ? idesc_whole : idesc_half;
        if (!mbar_wait(&ctl.tempty[acc], acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * UMMA_N);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&ctl.full[stage], phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * P_STAGE_BYTES);
          const uint32_t b_addr = a_addr + P_A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BKB / 32; ++kk) {
            const uint64_t da = sw128_kmajor_desc(a_addr + kk * 32);
            const uint64_t db = sw128_kmajor_desc(b_addr + kk * 32);
            if constexpr (kQ8)
              mma_e4m3_ss_pair(d_tmem, da, db, idesc, (kb | kk) != 0);
            else
              mma_bf16_ss_pair(d_tmem, da, db, idesc, (kb | kk) != 0);
          }
          mma_commit_pair_mc(&ctl.empty[stage], 0x3);
          if (++stage == P_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair_mc(&ctl.tfull[acc], 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      // Every issued MMA has completed before TMEM is released.
      mma_commit_pair(&ctl.drain);
      int never = 0;
      mbar_wait(&ctl.drain, 0, &never, p.status);
    }
  } else {
    // -------------------------------------------------- epilogue (warps 2 ..)
    const int q = warp & 3, part = (warp - 2) >> 2;
    constexpr int kParts = kEpiWarps / 4;
    const uint32_t tempty0 = mapa_shared(smem_u32(&ctl.tempty[0]), 0);
    float* stg = reinterpret_cast<float*>(smem + P_STAGES * P_STAGE_BYTES + kPairCtlBytes +
                                          (warp - 2) * (PairGeo<MODE, kQ8>::kStageTile +
                                                        PairGeo<MODE, kQ8>::kScales));
    float* sws = stg + PairGeo<MODE, kQ8>::kStageTile / 4;
    int acc = 0;
    uint32_t acc_phase = 0;
    // An item's rows and columns for this warp.
    struct Part {
      bool valid;
      int64_t prow;
      int n0, w, c0, c1;
      EpiRow own;
    };
    auto part_of = [&](int tile, int half) {
      Part o;
      int e, m_blk, n_blk;
      coords(tile, e, m_blk, n_blk);
      const int row_local = m_blk * PM + static_cast<int>(rank) * BM + q * 32 + lane;
      o.valid = row_local < ctl.off[e + 1] - ctl.off[e];
      o.prow = static_cast<int64_t>(ctl.off[e]) + row_local;
      o.w = half < 0 ? kTileN : kTileN / 2;
      o.n0 = n_blk * kTileN + (half < 0 ? 0 : half * o.w);
      o.c0 = part * (o.w / 32) / kParts;
      o.c1 = (part + 1) * (o.w / 32) / kParts;
      o.own = epilogue_row<MODE, kQ8>(p, o.valid, o.prow, e, o.n0, o.c0, o.c1);
      return o;
    };
    // In 8 bits the next item's slots, weights and scales are on their way while
    // this item's accumulator is stored.
    int tile, half;
    Part next;
    if (kQ8 && item(0, tile, half)) next = part_of(tile, half);
    for (int j = 0; item(j, tile, half); ++j) {
      Part cur;
      if (kQ8) cur = next;
      else cur = part_of(tile, half);
      if (!mbar_wait_warp(&ctl.tfull[acc], acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      if (kQ8 && item(j + 1, tile, half)) next = part_of(tile, half);
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * UMMA_N);
      epilogue_rows<MODE, kQ8>(p, t_row, cur.valid, cur.prow, cur.own, cur.n0, cur.w, cur.c0,
                               cur.c1, stg, sws);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(&ctl.tempty[acc]);
        else
          mbar_arrive_remote_relaxed(tempty0 + static_cast<uint32_t>(acc * sizeof(uint64_t)));
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA releases TMEM or exits while the other works
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// Swap-AB variant for few tokens per expert (decode): the weight rows are the
// MMA's M side (128 per tile) and the expert's tokens its N side (64 per
// tile), so a tile streams 128 x K of weights once and the tile count is
// E x N/128 x ceil(n_e / 64) -- enough tiles to cover the SMs even when every
// expert has only a handful of tokens. The kernel is bound by HBM, not by
// the SM count, so the grid is sized to give every CTA the same number of
// tiles (320 tiles: 107 CTAs of 3 tiles, not 148 CTAs and a partial wave). Same
// output as the Out / in-projection epilogue: out[token][n] = r * acc (bf16,
// k == 1) or per slot in float32; in 8 bits also Conv+Gate's.
constexpr int SW_BM = 128;                     // weight rows per tile (MMA M)
constexpr int SW_BN = 64;                      // tokens per tile (MMA N)
constexpr int SW_MAX_STAGES = 8;
constexpr int SW_A_BYTES = SW_BM * BK * 2;     // 16 KB of weights
constexpr int SW_B_BYTES = SW_BN * BK * 2;     // 8 KB of tokens
// Conv+Gate (8-bit products only): a stage holds the tile's W_in and W_g rows
// and an accumulator is u next to z, 64 tokens each.
template <int MODE>
struct SwapGeo {
  static constexpr bool kGate = (MODE == kEpiGateH || MODE == kEpiGateSlots);
  static constexpr int kStages = kGate ? 5 : SW_MAX_STAGES;
  static constexpr int kStageBytes = (kGate ? 2 : 1) * SW_A_BYTES + SW_B_BYTES;
  static constexpr int kAccCols = (kGate ? 2 : 1) * SW_BN;
  static constexpr uint32_t kTmemCols = 2 * kAccCols;
};

struct SwapCtl {
  uint64_t full[SW_MAX_STAGES];
  uint64_t empty[SW_MAX_STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int tile_start[kMaxExperts + 1];
  int off[kMaxExperts + 1];
  int tt[kMaxExperts];  // token tiles per expert
};

template <int MODE>
constexpr size_t kSwapSmemBytes =
    SwapGeo<MODE>::kStages * SwapGeo<MODE>::kStageBytes + sizeof(SwapCtl) + 1024;

// Output row, router weight and (8 bits) row scale of one token of the tile, for
// the lane that holds it (one token per lane, so the slot, weight and scale loads
// of a chunk of 32 tokens are issued together rather than one dependent chain per
// store).
template <int MODE, bool kQ8>
__device__ __forceinline__ void swap_token(const Params& p, int64_t prow, bool valid, int& orow,
                                           float& r, float& sa) {
  orow = 0;
  r = sa = 0.f;
  if (valid) {
    const int slot = MODE == kEpiGateH ? 0 : static_cast<int>(slot_of(p, prow));
    // no routing weights: r = 1
    r = !SwapGeo<MODE>::kGate && p.topk_w ? p.topk_w[slot] : 1.f;
    if (kQ8) sa = p.a_scale[prow];
    orow = MODE == kEpiGateH        ? static_cast<int>(prow)
           : MODE == kEpiScaleToken ? slot / p.k
                                    : slot;
  }
}

// kDense: the small-batch form without a dispatch (T <= 64 tokens, one token
// block). Every expert's weight tiles meet all T tokens, which the producer
// loads in token order; the routing decides only which results are kept: for
// token t and expert e, the epilogue stores r * acc where e is one of t's
// selected experts and nothing otherwise. The weights stream once either
// way (each expert's tiles for its single token block), and since nothing
// before the epilogue depends on the routing, the kernel is launched as a
// programmatic dependent of the router and only its epilogue waits for it.
template <int MODE, bool kDense, bool kQ8>
__global__ void __launch_bounds__(kThreads, 1)
    tc_swap_gemm_kernel(const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmW1,
                        const __grid_constant__ CUtensorMap tmX, const Params p) {
  constexpr bool kGate = SwapGeo<MODE>::kGate;
  constexpr int SW_STAGES = SwapGeo<MODE>::kStages;
  constexpr int SW_STAGE_BYTES = SwapGeo<MODE>::kStageBytes;
  constexpr int kXOff = SW_STAGE_BYTES - SW_B_BYTES;  // the tokens' rows in a stage
  constexpr int kAccCols = SwapGeo<MODE>::kAccCols;
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned base, kept as a shared-memory pointer (an offset into
  // the shared array, not an integer round-trip) so accesses stay LDS/STS.
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  SwapCtl& ctl = *reinterpret_cast<SwapCtl*>(smem + SW_STAGES * SW_STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  const int n_wt = p.N / SW_BM;  // weight-row tiles per expert

  // Set-up that needs no routing: barriers, TMEM, tensor maps. The kernel is
  // launched as a programmatic dependent of the dispatch, so this overlaps
  // the router and the dispatch. (An L2 prefetch of each CTA's first weight
  // tile here measured no gain on the decode step: 79.9 us either way.)
  if (threadIdx.x == 0) {
    for (int s = 0; s < SW_STAGES; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&ctl.tfull[a], 1);
      mbar_init(&ctl.tempty[a], 4);
    }
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem_base, SwapGeo<MODE>::kTmemCols);
    tmem_relinquish();
  }
  if (!kDense) {
    pdl_wait();  // the routing (offsets, sorted rows, weights) is complete from here
    for (int i = threadIdx.x; i <= E; i += kThreads) ctl.off[i] = offset_of(p, i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int run = 0;
    for (int e = 0; e < E; ++e) {
      // dense: one block of all (<= 64) tokens per expert, in token order
      const int tt = kDense ? 1 : (ctl.off[e + 1] - ctl.off[e] + SW_BN - 1) / SW_BN;
      ctl.tt[e] = tt;
      ctl.tile_start[e] = run;
      run += tt * n_wt;
    }
    ctl.tile_start[E] = run;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem_base;
  const int total = ctl.tile_start[E];
  const int KB = (p.K + kBK<kQ8> - 1) / kBK<kQ8>;
  volatile int* abort_flag = &ctl.abort;
  // tile -> (expert, weight-row block, token block); weight-row blocks vary
  // fastest so that CTAs running together share the expert's token rows.
  auto coords = [&](int tile, int& e, int& w_blk, int& t_blk) {
    e = 0;
    while (tile >= ctl.tile_start[e + 1]) ++e;
    const int local = tile - ctl.tile_start[e];
    t_blk = local / n_wt;
    w_blk = local - t_blk * n_wt;
  };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, last_par = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        int e, w_blk, t_blk;
        coords(tile, e, w_blk, t_blk);
        const int n0 = w_blk * SW_BM;
        const int r0 = kDense ? 0 : ctl.off[e] + t_blk * SW_BN;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&ctl.empty[stage], phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * SW_STAGE_BYTES;
          mbar_arrive_expect_tx(&ctl.full[stage], SW_STAGE_BYTES);
          if (kDense && p.w_tiled)
            tma_load_5d(sa, &tmW, &ctl.full[stage], 0, 0, kb, w_blk, e);
          else
            tma_load_3d(sa, &tmW, &ctl.full[stage], kb * kBK<kQ8>, n0, e);
          if (kGate)
            tma_load_3d(sa + SW_A_BYTES, &tmW1, &ctl.full[stage], kb * kBK<kQ8>, n0, e);
          tma_load_2d(sa + kXOff, &tmX, &ctl.full[stage], kb * kBK<kQ8>, r0);
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == SW_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      int never = 0;
      for (int s = 0; s < SW_STAGES; ++s)
        if ((issued >> s) & 1u) mbar_wait(&ctl.full[s], (last_par >> s) & 1u, &never, p.status);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = kQ8 ? idesc_e4m3_f32(SW_BM, SW_BN) : idesc_bf16_f32(SW_BM, SW_BN);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        if (!mbar_wait(&ctl.tempty[acc], acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAccCols);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&ctl.full[stage], phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * SW_STAGE_BYTES);
          const uint32_t b_addr = a_addr + kXOff;
#pragma unroll
          for (int kk = 0; kk < BKB / 32; ++kk) {
            const uint64_t da = sw128_kmajor_desc(a_addr + kk * 32);
            const uint64_t db = sw128_kmajor_desc(b_addr + kk * 32);
            if constexpr (kQ8)
              mma_e4m3_ss(d_tmem, da, db, idesc, (kb | kk) != 0);
            else
              mma_bf16_ss(d_tmem, da, db, idesc, (kb | kk) != 0);
            if constexpr (kGate)
              mma_e4m3_ss(d_tmem + SW_BN, sw128_kmajor_desc(a_addr + SW_A_BYTES + kk * 32), db,
                          idesc, (kb | kk) != 0);
          }
          mma_commit(&ctl.empty[stage]);
          if (++stage == SW_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(&ctl.tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      mma_commit(&ctl.drain);
      int never = 0;
      mbar_wait(&ctl.drain, 0, &never, p.status);
    }
  } else {
    const int q = warp & 3;
    int acc = 0;
    uint32_t acc_phase = 0;
    if (kDense) pdl_wait();  // the router's topk_idx / topk_w are complete from here
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      int e, w_blk, t_blk;
      coords(tile, e, w_blk, t_blk);
      int nv;  // token columns of the tile that may be stored
      int orow[2];
      float rw[2], sa[2];
      bool keep[2] = {true, true};
      if (kDense) {
        nv = static_cast<int>(p.R < SW_BN ? p.R : SW_BN);  // all T tokens, one block
        // column c*32 + lane is token t; kept where e is one of its experts
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int t = 32 * c + lane;
          keep[c] = false;
          orow[c] = 0;
          rw[c] = 0.f;
          if (t < nv)
            for (int j = 0; j < p.k; ++j) {
              const int64_t slot = static_cast<int64_t>(t) * p.k + j;
              if (p.topk_idx[slot] == e) {
                keep[c] = true;
                rw[c] = p.topk_w[slot];
                orow[c] = MODE == kEpiScaleToken ? t : static_cast<int>(slot);
              }
            }
        }
      } else {
        const int n_e = ctl.off[e + 1] - ctl.off[e];
        nv = min(SW_BN, n_e - t_blk * SW_BN);  // valid token columns, >= 1
        // token info first: its loads overlap the wait for the accumulator
        const int64_t prow0 = static_cast<int64_t>(ctl.off[e]) + t_blk * SW_BN;
        swap_token<MODE, kQ8>(p, prow0 + lane, lane < nv, orow[0], rw[0], sa[0]);
        swap_token<MODE, kQ8>(p, prow0 + 32 + lane, 32 + lane < nv, orow[1], rw[1], sa[1]);
      }
      if (!mbar_wait_warp(&ctl.tfull[acc], acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kAccCols);
      const int n = w_blk * SW_BM + q * 32 + lane;  // this thread's output column
      const float sw = kQ8 ? p.w0_scale[static_cast<int64_t>(e) * p.N + n] : 1.f;
      const float sw1 = kGate ? p.w1_scale[static_cast<int64_t>(e) * p.N + n] : 1.f;
#pragma unroll
      for (int c = 0; c < SW_BN / 32; ++c) {
        if (32 * c < nv) {  // warp-uniform
          uint32_t a[32], z[kGate ? 32 : 1];
          tmem_ld32(t_row + c * 32, a);
          if constexpr (kGate) tmem_ld32(t_row + SW_BN + c * 32, z);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (32 * c + j < nv) {  // warp-uniform
              if constexpr (kGate) {
                const int64_t i =
                    static_cast<int64_t>(__shfl_sync(0xffffffffu, orow[c], j)) * p.N + n;
                const float row_scale = __shfl_sync(0xffffffffu, sa[c], j);
                const float uv = __uint_as_float(a[j]) * row_scale * sw;
                const float zv = __uint_as_float(z[j]) * row_scale * sw1;
                if (MODE == kEpiGateH) {
                  static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(silu_gate(uv, zv));
                } else {
                  static_cast<float*>(p.out)[i] = uv;
                  static_cast<float*>(p.out)[p.R * p.N + i] = zv;
                }
                continue;
              }
              const int o = __shfl_sync(0xffffffffu, orow[c], j);
              float v = __uint_as_float(a[j]);
              if (kQ8) v = v * __shfl_sync(0xffffffffu, sa[c], j) * sw;
              v *= __shfl_sync(0xffffffffu, rw[c], j);
              const bool kept = __shfl_sync(0xffffffffu, keep[c] ? 1 : 0, j) != 0;
              const int64_t i = static_cast<int64_t>(o) * p.N + n;
              if (kept) {
                if (MODE == kEpiScaleToken)
                  static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
                else
                  static_cast<float*>(p.out)[i] = v;
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, SwapGeo<MODE>::kTmemCols);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Tensor map over a row-major [rows][K] matrix (or [E][rows][K] when
// experts > 0) of bf16 or, kQ8, of 8-bit codes: a box of box_rows rows of 128
// bytes, 128-byte swizzle.
template <bool kQ8 = false>
bool make_map(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int experts,
              int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(experts > 0 ? experts : 1)};
  const int64_t es = kQ8 ? 1 : 2;
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(K * es), static_cast<cuuint64_t>(K * es * rows)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(kBK<kQ8>), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const cuuint32_t rank = experts > 0 ? 3 : 2;
  CUresult r = fn(m, kQ8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                  const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int MODE, bool kQ8>
cudaError_t launch_pair_mode(const CUtensorMap& a, const CUtensorMap& b0, const CUtensorMap& b1,
                             const CUtensorMap& b0h, const CUtensorMap& b1h, const Params& p,
                             int64_t max_tiles, cudaStream_t stream) {
  auto kern = tc_pair_gemm_kernel<MODE, kQ8>;
  constexpr size_t kPairSmemBytes = pair_smem_bytes<MODE, kQ8>();
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kPairSmemBytes));
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // 8-bit products: the set-up runs while the kernel before finishes (1537 tokens,
  // top-2, K 2048, N 1024 over 16 experts and the sum of the slots: 23.3 -> 21.2 us)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(PairGeo<MODE, kQ8>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = kPairSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = kQ8 ? 2 : 1;
  // Co-resident pairs on this device (one CTA per SM), cached per device.
  static int pairs_cache[64] = {0};
  int dev = 0;
  err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  int pairs = (dev < 64) ? pairs_cache[dev] : 0;
  if (pairs == 0) {
    cfg.gridDim = dim3(2 * 64, 1, 1);
    err = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
    if (err != cudaSuccess) return err;
    if (pairs <= 0) return cudaErrorNotSupported;
    if (dev < 64) pairs_cache[dev] = pairs;
  }
  const int64_t n = std::min<int64_t>(pairs, max_tiles);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * n), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, a, b0, b1, b0h, b1h, p);
}

// The grouped GEMM in bf16, or in 8 bits with the rows' and features' scales.
template <bool kQ8>
cudaError_t launch_grouped(int mode, const void* a_sorted, const float* a_scale, int64_t R, int K,
                           const void* w0, const float* w0_scale, const void* w1,
                           const float* w1_scale, int N, int E, int k, const int32_t* offsets,
                           const int32_t* sorted_slot, const float* topk_w, void* out,
                           int* status, cudaStream_t stream) {
  constexpr int kAlign = kQ8 ? 16 : 8;  // elements of 16 bytes
  const bool gate = (mode == kEpiGateH || mode == kEpiGateSlots);
  const int tile_n = gate ? 128 : 256;
  // Few tokens (decode): the swap-AB kernel streams every weight tile once.
  if ((kQ8 || !gate) && R <= (kQ8 ? kSwapMaxRowsPerExpertQ8 * E : kSwapMaxRows) &&
      N % SW_BM == 0 && K % kAlign == 0 && E <= kMaxExperts) {
    if (R == 0) return cudaSuccess;
    CUtensorMap tw, tw1, tx;
    if (!make_map<kQ8>(&tw, w0, K, N, E, SW_BM)) return cudaErrorInvalidValue;
    tw1 = tw;
    if (gate && !make_map<kQ8>(&tw1, w1, K, N, E, SW_BM)) return cudaErrorInvalidValue;
    if (!make_map<kQ8>(&tx, a_sorted, K, R, 0, SW_BN)) return cudaErrorInvalidValue;
    Params p{};
    p.a_scale = a_scale;
    p.w0_scale = w0_scale;
    p.w1_scale = w1_scale;
    p.offsets = offsets;
    p.sorted_slot = sorted_slot;
    p.topk_w = topk_w;
    p.out = out;
    p.R = R;
    p.K = K;
    p.N = N;
    p.E = E;
    p.k = k;
    p.status = status;
    // Upper bound of the tile count (the exact count depends on the routing,
    // read on the device); every CTA gets ceil(tiles / SMs) tiles.
    const int64_t max_tiles = ((R + SW_BN - 1) / SW_BN + E) * static_cast<int64_t>(N / SW_BM);
    const int64_t tiles_ub = std::min<int64_t>(
        max_tiles, static_cast<int64_t>(E) * (N / SW_BM) * ((R + SW_BN - 1) / SW_BN));
    const int64_t sms = device_sm_count();
    const int64_t per_cta = (tiles_ub + sms - 1) / sms;
    const int grid = static_cast<int>(std::min<int64_t>(sms, (tiles_ub + per_cta - 1) / per_cta));
    auto kern = (mode == kEpiScaleToken) ? tc_swap_gemm_kernel<kEpiScaleToken, false, kQ8>
                                         : tc_swap_gemm_kernel<kEpiScaleSlots, false, kQ8>;
    size_t smem = kSwapSmemBytes<kEpiScaleToken>;
    if constexpr (kQ8) {
      if (gate) {
        kern = (mode == kEpiGateH) ? tc_swap_gemm_kernel<kEpiGateH, false, true>
                                   : tc_swap_gemm_kernel<kEpiGateSlots, false, true>;
        smem = kSwapSmemBytes<kEpiGateH>;
      }
    }
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    // Programmatic dependent launch: the set-up runs
    // while the kernel before (the dispatch) finishes.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tw, tw1, tx, p);
  }
  if (K % kAlign != 0 || N % 128 != 0 || E > kMaxExperts || R >= (int64_t(1) << 31))
    return cudaErrorInvalidValue;
  if (R == 0) return cudaSuccess;
  CUtensorMap ta, tb0, tb1, tb0h, tb1h;
  {
    // B maps: boxes of 128 rows (whole tiles) and 64 rows (half tiles)
    if (!make_map<kQ8>(&ta, a_sorted, K, R, 0, BM)) return cudaErrorInvalidValue;
    if (!make_map<kQ8>(&tb0, w0, K, N, E, 128)) return cudaErrorInvalidValue;
    if (!make_map<kQ8>(&tb0h, w0, K, N, E, 64)) return cudaErrorInvalidValue;
    if (gate) {
      if (!make_map<kQ8>(&tb1, w1, K, N, E, 128)) return cudaErrorInvalidValue;
      if (!make_map<kQ8>(&tb1h, w1, K, N, E, 64)) return cudaErrorInvalidValue;
    } else {
      tb1 = tb0;
      tb1h = tb0h;
    }
    Params p{};
    p.offsets = offsets;
    p.sorted_slot = sorted_slot;
    p.topk_w = topk_w;
    p.out = out;
    p.R = R;
    p.K = K;
    p.N = N;
    p.E = E;
    p.k = k;
    p.n_tiles_n = (N + tile_n - 1) / tile_n;
    p.a_scale = a_scale;
    p.w0_scale = w0_scale;
    p.w1_scale = w1_scale;
    p.status = status;
    const int64_t max_tiles = ((R + PM - 1) / PM + E) * static_cast<int64_t>(p.n_tiles_n);
    switch (mode) {
      case kEpiGateH:
        return launch_pair_mode<kEpiGateH, kQ8>(ta, tb0, tb1, tb0h, tb1h, p, max_tiles, stream);
      case kEpiGateSlots:
        return launch_pair_mode<kEpiGateSlots, kQ8>(ta, tb0, tb1, tb0h, tb1h, p, max_tiles, stream);
      case kEpiScaleToken:
        return launch_pair_mode<kEpiScaleToken, kQ8>(ta, tb0, tb1, tb0h, tb1h, p, max_tiles, stream);
      case kEpiScaleSlots:
        return launch_pair_mode<kEpiScaleSlots, kQ8>(ta, tb0, tb1, tb0h, tb1h, p, max_tiles, stream);
      default:
        return cudaErrorInvalidValue;
    }
  }
}

}  // namespace

bool make_tile_map(CUtensorMap* m, const void* base, int bytes, int64_t kb, int64_t tiles,
                   int box_kb, int box_tiles) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(bytes / 4), static_cast<cuuint64_t>(kb),
                              static_cast<cuuint64_t>(tiles)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(bytes),
                                 static_cast<cuuint64_t>(bytes) * static_cast<cuuint64_t>(kb)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(bytes / 4), static_cast<cuuint32_t>(box_kb),
                             static_cast<cuuint32_t>(box_tiles)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_tc_grouped_gemm(int mode, const void* a_sorted, int64_t R, int K,
                                   const void* w0, const void* w1, int N, int E, int k,
                                   const int32_t* offsets, const int32_t* sorted_slot,
                                   const float* topk_w, void* out, int* status,
                                   cudaStream_t stream) {
  return launch_grouped<false>(mode, a_sorted, nullptr, R, K, w0, nullptr, w1, nullptr, N, E, k,
                               offsets, sorted_slot, topk_w, out, status, stream);
}

cudaError_t launch_tc_grouped_gemm_q8(int mode, const void* a_sorted, const float* a_scale,
                                      int64_t R, int K, const void* w0, const float* w0_scale,
                                      const void* w1, const float* w1_scale, int N, int E, int k,
                                      const int32_t* offsets, const int32_t* sorted_slot,
                                      const float* topk_w, void* out, int* status,
                                      cudaStream_t stream) {
  return launch_grouped<true>(mode, a_sorted, a_scale, R, K, w0, w0_scale, w1, w1_scale, N, E, k,
                              offsets, sorted_slot, topk_w, out, status, stream);
}

cudaError_t launch_tc_dense_small(int mode, const void* x, int64_t T, int K, const void* w, int N,
                                  int E, int k, const int32_t* topk_idx, const float* topk_w,
                                  void* out, bool w_tiled, int* status, cudaStream_t stream) {
  if (T <= 0) return cudaSuccess;
  if (T > SW_BN || N % SW_BM != 0 || K % 8 != 0 || E > kMaxExperts) return cudaErrorInvalidValue;
  if (w_tiled && K % BK != 0) return cudaErrorInvalidValue;
  CUtensorMap tw, tx;
  if (w_tiled) {
    // [E][N/128][K/64][128][64]: a box of one whole 128 x 64 tile (16 KB)
    auto fn = encode_fn();
    if (!fn) return cudaErrorInvalidValue;
    const cuuint64_t kb = static_cast<cuuint64_t>(K / BK), nt = static_cast<cuuint64_t>(N / SW_BM);
    const cuuint64_t tile_bytes = static_cast<cuuint64_t>(SW_BM) * BK * 2;
    cuuint64_t dims[5] = {static_cast<cuuint64_t>(BK), static_cast<cuuint64_t>(SW_BM), kb, nt,
                          static_cast<cuuint64_t>(E)};
    cuuint64_t strides[4] = {static_cast<cuuint64_t>(BK) * 2, tile_bytes, tile_bytes * kb,
                             tile_bytes * kb * nt};
    cuuint32_t box[5] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(SW_BM), 1, 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    if (fn(&tw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(w), dims, strides, box,
           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  } else if (!make_map(&tw, w, K, N, E, SW_BM)) {
    return cudaErrorInvalidValue;
  }
  if (!make_map(&tx, x, K, T, 0, SW_BN)) return cudaErrorInvalidValue;
  Params p{};
  p.topk_idx = topk_idx;
  p.w_tiled = w_tiled ? 1 : 0;
  p.topk_w = topk_w;
  p.out = out;
  p.R = T;  // token rows (in token order)
  p.K = K;
  p.N = N;
  p.E = E;
  p.k = k;
  p.status = status;
  // every CTA gets the same number of tiles (E x N/128 tiles in all)
  const int64_t tiles = static_cast<int64_t>(E) * (N / SW_BM);
  const int64_t sms = device_sm_count();
  const int64_t per_cta = (tiles + sms - 1) / sms;
  const int grid = static_cast<int>(std::min<int64_t>(sms, (tiles + per_cta - 1) / per_cta));
  auto kern = (mode == kEpiScaleToken) ? tc_swap_gemm_kernel<kEpiScaleToken, true, false>
                                       : tc_swap_gemm_kernel<kEpiScaleSlots, true, false>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSwapSmemBytes<kEpiScaleToken>));
  if (err != cudaSuccess) return err;
  // a programmatic dependent of the router: the weight streaming and the
  // MMAs run while the router finishes; the epilogue waits for it
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSwapSmemBytes<kEpiScaleToken>;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tw, tw, tx, p);
}

}  // namespace rom
