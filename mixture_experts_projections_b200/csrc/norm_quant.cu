// The norm in front of a block and the 8-bit rows its experts read.
//
//   rom_add_rmsnorm       s = x + res (stored in res's type),
//                         rstd = 1 / sqrt(mean(s^2) + eps), y = s * rstd * w,
//                         y in x's type and / or as 8-bit rows
//   rom_add_rmsnorm_bwd   with g = dy * w:
//                         ds = dres_out + rstd * (g - s * rstd^2 * mean(g * s)),
//                         dw = sum_t dy * s * rstd
//   rom_quant_rows        8-bit rows of a matrix
//
// 8-bit rows: e4m3 with one float32 scale per row, scale = max(a, 2^-100) / 448
// with a = max |v| of the row, q = e4m3(v * (448 / max(a, 2^-100))), so that the
// row's largest value is e4m3's largest (448) and q * scale stands for v. The
// floor keeps the scale and its reciprocal normal numbers; a row of zeros is
// zeros. A row that holds an infinity or a NaN has no such scale: its codes and
// its scale are NaN, so that every product with it is NaN.
//
// The norm is that of s as it is stored: the backward has only the stored s,
// and so differentiates the function that ran. All sums are float32.
//
// All three are bound by memory. A row stays in registers between its single
// read and its writes: one CTA per row, 8 columns (16 bytes of bf16) per
// thread and step, V steps; short rows take a warp or a part of one. The choice
// goes by the row's length alone, so a row's result does not depend on the batch.
// 16384 x 2048 bf16 with a float32 residual and 8-bit rows: 66 us in a graph (68 as
// called from Python), the 437 MB at the measured copy rate; the gradient of 32768 x
// 2560 bf16 with a bf16 residual: 134 us (128).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "rom_internal.cuh"
#include "sm100_ptx.cuh"

namespace rom {
namespace {

constexpr float kE4m3Max = 448.0f;
// Rows of 520 to 2048 columns that a CTA of the backward goes through at a time:
// as many as 512 threads hold, up to this many (of shorter rows, 8 warps' worth).
constexpr int kNormBwdGroups = 4;
// Most shared memory of a CTA of the backward that stages its rows: 3 pieces of 16
// bytes, 4 steps, 512 threads.
constexpr int kNormBwdStagedBytes = 16 * 3 * 4 * 512;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100

// 8 elements as they are stored, and their values.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void values(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x), v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z), v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void values(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {  // all but the last N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The value that storing v in T leaves.
__device__ __forceinline__ float as_stored(float v, const float*) { return v; }
__device__ __forceinline__ float as_stored(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

// A row's threads: kLanes of a warp (8, 16 or 32; blockDim = (kLanes, rows)), the
// whole CTA (0), or
// (kGroups) one of its blockDim.y groups with a named barrier each. Sums and
// maxima over them come back in every thread; the order of the additions is
// fixed. `red` holds one value per warp and is written once per kernel (or
// between barriers of the caller).
template <int kLanes, bool kGroups = false>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = (kLanes ? kLanes : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (kLanes) return v;
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  if (kGroups)
    named_barrier_sync(1 + threadIdx.y, blockDim.x);
  else
    __syncthreads();
  float s = 0.f;
  for (int i = 0; i < nw; ++i) s += red[i];
  return s;
}
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  if (kLanes == 0 || kLanes == 32) {
    v = __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  if (kLanes) return v;
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  uint32_t s = 0;
  for (int i = 0; i < nw; ++i) s = max(s, red[i]);
  return s;
}

// Bits of |v|: they order as the values do, and a NaN above all of them.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The row's scale and the factor of its codes from the bits of max |v|.
__device__ __forceinline__ void row_scale(uint32_t amax_bits, float& scale, float& inv) {
  if (amax_bits >= 0x7f800000u) {
    scale = inv = __uint_as_float(0x7fffffffu);
  } else {
    const float a = fmaxf(__uint_as_float(amax_bits), kAmaxFloor);
    scale = __fdiv_rn(a, kE4m3Max);
    inv = __fdiv_rn(kE4m3Max, a);
  }
}

// 8 codes. |v * inv| is at most 448 (1 + 2^-22), which rounds to 448.
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <typename XT, typename RT, int V, int kLanes>
__global__ void __launch_bounds__(512)
    add_rmsnorm_kernel(const XT* x, const RT* res, int64_t T, int D,
                                   const float* __restrict__ w, float eps, RT* res_out, XT* y,
                                   uint8_t* __restrict__ y8, float* __restrict__ y_scale,
                                   float* __restrict__ rstd_out) {
  __shared__ float red[32];
  __shared__ uint32_t redm[32];
  const int64_t row =
      kLanes ? blockIdx.x * static_cast<int64_t>(blockDim.y) + threadIdx.y : blockIdx.x;
  const int cols = kLanes && row >= T ? 0 : D;  // no row: no columns
  const int step = kLanes ? kLanes : blockDim.x;
  const int64_t base = row * D;
  float s[V][8];
  float sum = 0.f;
  pdl_wait();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * step) * 8;
    if (c < cols) {
      load8(x + base + c, s[i]);
      if (res) {
        float r[8];
        load8(res + base + c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[i][j] = as_stored(s[i][j], res_out);
        sum = fmaf(s[i][j], s[i][j], sum);
      }
    }
  }
  sum = row_sum<kLanes>(sum, red);
  const float rstd = rsqrtf(sum / static_cast<float>(D) + eps);
  if (threadIdx.x == 0 && cols && rstd_out) rstd_out[row] = rstd;
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * step) * 8;
    if (c < cols) {
      if (res_out) store8(res_out + base + c, s[i]);
      float wv[8];
      load8(w + c, wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[i][j] = s[i][j] * rstd * wv[j];
        amax = max(amax, abs_bits(s[i][j]));
      }
      if (y) store8(y + base + c, s[i]);
    }
  }
  if (y8) {
    amax = row_max<kLanes>(amax, redm);
    float scale, inv;
    row_scale(amax, scale, inv);
    if (threadIdx.x == 0 && cols) y_scale[row] = scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (c < cols) store_codes(y8 + base + c, s[i], inv);
    }
  }
}

// Persistent CTAs; a row is on its way while the one before it is converted
// (16384 x 4096 bf16: 36 us, 50 with a CTA per row and one step per thread; 31 by
// the bytes).
template <typename XT, int V, int kLanes>
__global__ void __launch_bounds__(512)
    quant_rows_kernel(const XT* __restrict__ x, int64_t rows, int D, uint8_t* __restrict__ q,
                      float* __restrict__ scale_out) {
  __shared__ uint32_t redm[2][32];
  const int step = kLanes ? kLanes : blockDim.x;
  const int64_t row0 =
      kLanes ? blockIdx.x * static_cast<int64_t>(blockDim.y) + threadIdx.y : blockIdx.x;
  const int64_t row_step = kLanes ? gridDim.x * static_cast<int64_t>(blockDim.y) : gridDim.x;
  Raw8<XT> next[V];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (row < rows && c < D) next[i] = load_raw(x + row * D + c);
    }
  };
  pdl_wait();
  fetch(row0);
  // a warp's rows go on together
  const int after = kLanes ? threadIdx.y % (32 / (kLanes ? kLanes : 32)) : 0;
  int buf = 0;
  for (int64_t row = row0; row - after < rows; row += row_step, buf ^= 1) {
    const int cols = kLanes && row >= rows ? 0 : D;  // no row: no columns
    float s[V][8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (c < cols) {
        values(next[i], s[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(s[i][j]));
      }
    }
    fetch(row + row_step);
    amax = row_max<kLanes>(amax, redm[buf]);
    float scale, inv;
    row_scale(amax, scale, inv);
    if (threadIdx.x == 0 && cols) scale_out[row] = scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (c < cols) store_codes(q + row * D + c, s[i], inv);
    }
  }
}

// CTA b takes rows b, b + gridDim.x, ...; a thread's columns stay its own, so
// that it adds up their dw over its CTA's rows in registers. The CTA's sums go
// to row b of the workspace, and dw_reduce_kernel adds them in a fixed order: no
// atomics, the same result every time. Every input of the next row is on its way
// while the current row is summed, for up to two steps per thread, which have the
// registers for it (with its loads after the sum's barrier, and none ahead, the
// kernel took 179 us for 32768 x 2560 bf16 where the bytes take 128). Longer rows
// of a bf16 stream wait in shared memory, each thread's own pieces (5000 x 16384:
// 138 us, 237 without; 125 by the bytes). Those of a float32 stream do not: all three
// inputs there leave the weights no L1 (bf16 rows of 16384 columns: 319 us, 282
// without; 200 by the bytes).
// Short rows leave room for several in a CTA, each with threads of its own
// (blockDim.y of them; 8, 16 or 32 lanes of a warp for up to 64, 128 or 512
// columns, kLanes): the CTA's sums of dw are theirs, added in order. With one row
// per CTA the workspace's 512 rows left SMs half empty: 11564 x 112 bf16 took 20 us
// (7 here), 20000 x 1024 57 (37).
// One step per thread of bf16 rows is held to 64 registers, for 1024 threads per
// SM: without the bound 20000 x 1024 took 48 us and 32768 x 2560 178 (136). Float32
// rows need more than those (32768 x 1024: 105 us, 125 with the bound), and so do a
// warp's rows with a float32 stream (131072 x 256: 93, 98).
template <typename XT, typename RT, int V, int kLanes, bool kGroups>
__global__ void __launch_bounds__(
    512, V == 1 && sizeof(XT) == 2 && !(kLanes && sizeof(RT) == 4) ? 2 : 1)
    add_rmsnorm_bwd_kernel(const XT* __restrict__ dy, const RT* dres_out,
                           const RT* __restrict__ s, int64_t T, int D,
                           const float* __restrict__ w, const float* __restrict__ rstd,
                           XT* __restrict__ dx, RT* dres, float* __restrict__ dw_part) {
  constexpr bool kAhead = V <= 2;                       // the next row in registers
  constexpr bool kStaged = !kAhead && sizeof(RT) == 2;  // or in shared memory
  constexpr bool kSeveral = kLanes || kGroups;
  __shared__ float red[2][kGroups ? kNormBwdGroups : 1][32];
  __shared__ float group_dw[kSeveral ? 4096 : 1];  // [blockDim.y][D]
  const int step = kLanes ? kLanes : blockDim.x;
  const int64_t row0 = kSeveral ? int64_t(blockIdx.x) * blockDim.y + threadIdx.y : blockIdx.x;
  const int64_t row_step = kSeveral ? int64_t(gridDim.x) * blockDim.y : gridDim.x;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  const float inv_d = 1.f / static_cast<float>(D);
  Raw8<XT> rg[kAhead ? V : 1];
  Raw8<RT> rs[kAhead ? V : 1], rd[kAhead ? V : 1];
  float r = 0.f;
  auto fetch = [&](int64_t row) {
    if (row < T) {
      const int64_t base = row * D;
      r = rstd[row];
#pragma unroll
      for (int i = 0; i < (kAhead ? V : 0); ++i) {
        const int c = (threadIdx.x + i * step) * 8;
        if (c < D) {
          rg[i] = load_raw(dy + base + c);
          rs[i] = load_raw(s + base + c);
          if (dres_out) rd[i] = load_raw(dres_out + base + c);
        }
      }
    }
  };
  // A thread's pieces of the next row's dy, s and dres_out: [3 V][blockDim.x].
  extern __shared__ uint4 staged[];
  auto piece = [&](int i) { return staged + i * blockDim.x + threadIdx.x; };
  auto copy = [&](int first, const auto* p, int64_t row) {
    if (row < T && p) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * step) * 8;
        if (c < D) cp_async16(piece(first + i), p + row * D + c);
      }
    }
  };
  auto copy_rows = [&](int64_t row) {
    if (row < T) r = rstd[row];
    copy(0, dy, row);
    copy(V, s, row);
    cp_async_commit();
  };
  auto copy_dres = [&](int64_t row) {
    copy(2 * V, dres_out, row);
    cp_async_commit();
  };
  pdl_wait();
  if constexpr (kAhead) {
    fetch(row0);
  } else if constexpr (kStaged) {
    copy_rows(row0);
    copy_dres(row0);
  }
  int buf = 0;
  // a warp's rows go on together
  const int after = kLanes ? threadIdx.y % (32 / (kLanes ? kLanes : 32)) : 0;
  for (int64_t row = row0; row - after < T; row += row_step, buf ^= 1) {
    const int64_t base = row * D;
    const int cols = kLanes && kLanes < 32 && row >= T ? 0 : D;
    if constexpr (kStaged) cp_async_wait<1>();
    if constexpr (!kAhead && !kStaged) fetch(row);
    const float rr = r;
    float g[V][8], sv[V][8];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (c < cols) {
        float wv[8];
        if constexpr (kAhead) {
          values(rg[i], g[i]);
          values(rs[i], sv[i]);
        } else if constexpr (kStaged) {
          load8(reinterpret_cast<const XT*>(piece(i)), g[i]);
          load8(reinterpret_cast<const RT*>(piece(V + i)), sv[i]);
        } else {
          load8(dy + base + c, g[i]);
          load8(s + base + c, sv[i]);
        }
        load8(w + c, wv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[i][j] = fmaf(g[i][j], sv[i][j] * rr, dw[i][j]);
          g[i][j] *= wv[j];
          dot = fmaf(g[i][j], sv[i][j], dot);
        }
      }
    }
    Raw8<RT> cd[kAhead ? V : 1];
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < V; ++i) cd[i] = rd[i];
      fetch(row + row_step);
    } else if constexpr (kStaged) {
      copy_rows(row + row_step);
    }
    // two buffers: a warp may still read this row's sums when another one
    // writes the next row's, never two rows on
    dot = row_sum<kLanes, kGroups>(dot, red[buf][kGroups ? threadIdx.y : 0]);
    const float k = rr * rr * (dot * inv_d);
    if constexpr (kStaged) cp_async_wait<1>();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (c < cols) {
        float d[8];
        if (dres_out) {
          if constexpr (kAhead)
            values(cd[i], d);
          else if constexpr (kStaged)
            load8(reinterpret_cast<const RT*>(piece(2 * V + i)), d);
          else
            load8(dres_out + base + c, d);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rr, fmaf(-sv[i][j], k, g[i][j]), d[j]);
        if (dx) store8(dx + base + c, d);
        if (dres) store8(dres + base + c, d);
      }
    }
    if constexpr (kStaged) copy_dres(row + row_step);
  }
  pdl_launch_dependents();  // the sum of the CTAs' dw may be set up
  if (kSeveral) {
    if (!dw_part) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (c < D) store8(group_dw + threadIdx.y * D + c, dw[i]);
    }
    __syncthreads();
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < D; c += blockDim.x * blockDim.y) {
      float t = group_dw[c];
      for (int i = 1; i < static_cast<int>(blockDim.y); ++i) t += group_dw[i * D + c];
      dw_part[static_cast<int64_t>(blockIdx.x) * D + c] = t;
    }
  } else if (dw_part) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * step) * 8;
      if (c < D) store8(dw_part + static_cast<int64_t>(blockIdx.x) * D + c, dw[i]);
    }
  }
}

// dw[c] = sum over the P rows of part, kCols columns per CTA: a warp reads 32 /
// kCols rows at a time, and the sums of 32 warps are added in a fixed order. 8
// columns (a 32-byte sector of a row) while that leaves at most two CTAs per SM,
// else 32: the gradient of 11564 x 112 takes 6.0 us with 8, 6.5 with 32; that of
// 4096 x 8192 bf16 with a float32 residual 96.9 with 8, 90.4 with 32 (82 by the bytes).
template <int kCols>
__global__ void __launch_bounds__(1024)
    dw_reduce_kernel(const float* __restrict__ part, int P, int D, float* __restrict__ dw) {
  constexpr int kRows = 32 / kCols;
  __shared__ float sum[32][kCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * kCols + lane % kCols;
  float v = 0.f;
  pdl_wait();  // the workspace is complete from here
  if (c < D) {
#pragma unroll 4
    for (int p = warp * kRows + lane / kCols; p < P; p += 32 * kRows)
      v += part[static_cast<int64_t>(p) * D + c];
  }
#pragma unroll
  for (int o = kCols; o < 32; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane < kCols) sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && lane < kCols && c < D) {
    float t = sum[0][lane];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += sum[i][lane];
    dw[c] = t;
  }
}

// Launches that may be set up while the kernel before on the stream finishes
// (every kernel here waits for it first): 517 x 1024 bf16 rows' gradient, 8.2 us
// with plain launches of its two kernels, 7.5 with the second one so.
template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), int64_t grid, dim3 block, size_t smem, cudaStream_t stream,
                   A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// Steps per thread (V), lanes of a warp (or 0) and the launch of one row's
// threads for D columns: rows of up to 64, 128 or 512 columns take a quarter, half
// or all of a warp, up to 4096 columns one step of a CTA with a thread for each 8
// columns, longer ones more steps. (With a warp for each row of 64 bf16 columns
// 262144 of them took 57 us, their gradient 73; 21 and 32 with a quarter.)
struct RowShape {
  int V;
  int lanes;
  dim3 block;
};
RowShape row_shape(int D, int fewest_steps = 1) {
  const int nvec = D / 8;
  if (nvec <= 64) {
    const int lanes = nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32;
    return {nvec <= 32 ? 1 : 2, lanes, dim3(lanes, 256 / lanes, 1)};
  }
  int V = fewest_steps;
  while (nvec > V * 512 && V < 4) V *= 2;
  const int threads = ((nvec + V - 1) / V + 31) / 32 * 32;
  return {V, 0, dim3(static_cast<unsigned>(threads), 1, 1)};
}

template <typename XT, typename RT>
cudaError_t add_rmsnorm(const void* x, const void* res, int64_t T, int D, const float* w,
                        float eps, void* res_out, void* y, void* y8, float* y_scale, float* rstd,
                        cudaStream_t stream) {
  const RowShape sh = row_shape(D);
  const unsigned grid = static_cast<unsigned>(sh.lanes ? (T + sh.block.y - 1) / sh.block.y : T);
  auto go = [&](auto kern) {
    return launch(kern, grid, sh.block, 0, stream, static_cast<const XT*>(x),
                  static_cast<const RT*>(res), T, D, w, eps, static_cast<RT*>(res_out),
                  static_cast<XT*>(y), static_cast<uint8_t*>(y8), y_scale, rstd);
  };
  if (sh.lanes)
    return sh.lanes == 8    ? go(add_rmsnorm_kernel<XT, RT, 1, 8>)
           : sh.lanes == 16 ? go(add_rmsnorm_kernel<XT, RT, 1, 16>)
           : sh.V == 1      ? go(add_rmsnorm_kernel<XT, RT, 1, 32>)
                            : go(add_rmsnorm_kernel<XT, RT, 2, 32>);
  switch (sh.V) {
    case 1:
      return go(add_rmsnorm_kernel<XT, RT, 1, 0>);
    case 2:
      return go(add_rmsnorm_kernel<XT, RT, 2, 0>);
    default:
      return go(add_rmsnorm_kernel<XT, RT, 4, 0>);
  }
}

template <typename XT>
cudaError_t quant_rows(const void* x, int64_t rows, int D, void* q, float* scale,
                       cudaStream_t stream) {
  const RowShape sh = row_shape(D, 2);
  const int64_t ctas = sh.lanes ? (rows + sh.block.y - 1) / sh.block.y : rows;
  const int threads = static_cast<int>(sh.block.x * sh.block.y);
  const int64_t grid =
      std::min<int64_t>(ctas, static_cast<int64_t>(device_sm_count()) * std::max(1, 2048 / threads));
  auto go = [&](auto kern) {
    return launch(kern, grid, sh.block, 0, stream, static_cast<const XT*>(x), rows, D,
                  static_cast<uint8_t*>(q), scale);
  };
  if (sh.lanes)
    return sh.lanes == 8    ? go(quant_rows_kernel<XT, 1, 8>)
           : sh.lanes == 16 ? go(quant_rows_kernel<XT, 1, 16>)
           : sh.V == 1      ? go(quant_rows_kernel<XT, 1, 32>)
                            : go(quant_rows_kernel<XT, 2, 32>);
  switch (sh.V) {
    case 1:
      return go(quant_rows_kernel<XT, 1, 0>);
    case 2:
      return go(quant_rows_kernel<XT, 2, 0>);
    default:
      return go(quant_rows_kernel<XT, 4, 0>);
  }
}

template <typename XT, typename RT>
cudaError_t add_rmsnorm_bwd(const void* dy, const void* dres_out, const void* s, int64_t T, int D,
                            const float* w, const float* rstd, void* dx, void* dres, float* dw,
                            float* ws, cudaStream_t stream) {
  const RowShape sh = row_shape(D);
  // Two rows or more per row's threads, up to 1024 threads per SM.
  const int per_row = static_cast<int>(sh.block.x);
  int rows_at_once = sh.lanes   ? static_cast<int>(sh.block.y)
                     : sh.V > 1 ? 1
                                : std::max(1, std::min(kNormBwdGroups, 512 / per_row));
  // Few rows: smaller CTAs on more SMs (64 x 2048 bf16: 4.3 us, 5.2 with four rows
  // to a CTA; of warp-sized rows they cost more parts of dw than they save).
  while (!sh.lanes && rows_at_once > 1 && T < rows_at_once * device_sm_count()) rows_at_once /= 2;
  const int threads = per_row * rows_at_once;
  const bool staged = sh.V > 2 && sizeof(RT) == 2;  // (its registers leave one CTA to an SM)
  const int per_sm = staged ? 1 : std::max(1, 1024 / threads);
  const int64_t grid =
      std::min<int64_t>({(T + 2 * rows_at_once - 1) / (2 * rows_at_once), kNormBwdMaxParts,
                         static_cast<int64_t>(device_sm_count()) * per_sm});
  const dim3 block(per_row, rows_at_once, 1);
  const size_t smem = staged ? sizeof(uint4) * 3 * sh.V * threads : 0;
  auto go = [&](auto kern) {
    if (smem) {
      // the limit belongs to the function, not to the launch: the same for every
      // width, or another thread's launch could find it too low for its own
      const cudaError_t e = cudaFuncSetAttribute(
          kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormBwdStagedBytes);
      if (e != cudaSuccess) return e;
    }
    return launch(kern, grid, block, smem, stream, static_cast<const XT*>(dy),
                  static_cast<const RT*>(dres_out), static_cast<const RT*>(s), T, D, w, rstd,
                  static_cast<XT*>(dx), static_cast<RT*>(dres), dw ? ws : nullptr);
  };
  cudaError_t err;
  if (sh.lanes)
    err = sh.lanes == 8    ? go(add_rmsnorm_bwd_kernel<XT, RT, 1, 8, false>)
          : sh.lanes == 16 ? go(add_rmsnorm_bwd_kernel<XT, RT, 1, 16, false>)
          : sh.V == 1      ? go(add_rmsnorm_bwd_kernel<XT, RT, 1, 32, false>)
                           : go(add_rmsnorm_bwd_kernel<XT, RT, 2, 32, false>);
  else if (rows_at_once > 1)
    err = go(add_rmsnorm_bwd_kernel<XT, RT, 1, 0, true>);
  else
    err = sh.V == 1   ? go(add_rmsnorm_bwd_kernel<XT, RT, 1, 0, false>)
          : sh.V == 2 ? go(add_rmsnorm_bwd_kernel<XT, RT, 2, 0, false>)
                      : go(add_rmsnorm_bwd_kernel<XT, RT, 4, 0, false>);
  if (err != cudaSuccess || !dw) return err;
  auto reduce = [&](auto kern, int cols) {
    return launch(kern, (D + cols - 1) / cols, dim3(1024), 0, stream, ws, static_cast<int>(grid), D,
                  dw);
  };
  return D / 8 <= 2 * device_sm_count() ? reduce(dw_reduce_kernel<8>, 8)
                                        : reduce(dw_reduce_kernel<32>, 32);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* x, bool x_bf16, const void* res, bool res_bf16,
                               int64_t T, int D, const float* w, float eps, void* res_out, void* y,
                               void* y8, float* y_scale, float* rstd, cudaStream_t stream) {
  if (x_bf16)
    return res_bf16 ? add_rmsnorm<__nv_bfloat16, __nv_bfloat16>(x, res, T, D, w, eps, res_out, y,
                                                                y8, y_scale, rstd, stream)
                    : add_rmsnorm<__nv_bfloat16, float>(x, res, T, D, w, eps, res_out, y, y8,
                                                        y_scale, rstd, stream);
  return add_rmsnorm<float, float>(x, res, T, D, w, eps, res_out, y, y8, y_scale, rstd, stream);
}

cudaError_t launch_add_rmsnorm_bwd(const void* dy, bool x_bf16, const void* dres_out,
                                   const void* s, bool res_bf16, int64_t T, int D, const float* w,
                                   const float* rstd, void* dx, void* dres, float* dw, float* ws,
                                   cudaStream_t stream) {
  if (x_bf16)
    return res_bf16 ? add_rmsnorm_bwd<__nv_bfloat16, __nv_bfloat16>(dy, dres_out, s, T, D, w, rstd,
                                                                    dx, dres, dw, ws, stream)
                    : add_rmsnorm_bwd<__nv_bfloat16, float>(dy, dres_out, s, T, D, w, rstd, dx,
                                                            dres, dw, ws, stream);
  return add_rmsnorm_bwd<float, float>(dy, dres_out, s, T, D, w, rstd, dx, dres, dw, ws, stream);
}

cudaError_t launch_quant_rows(const void* x, bool x_bf16, int64_t rows, int D, void* q,
                              float* scale, cudaStream_t stream) {
  return x_bf16 ? quant_rows<__nv_bfloat16>(x, rows, D, q, scale, stream)
                : quant_rows<float>(x, rows, D, q, scale, stream);
}

}  // namespace rom
