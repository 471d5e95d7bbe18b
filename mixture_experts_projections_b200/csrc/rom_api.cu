// C ABI of librom.so: argument validation, mode selection and launches.
// The declarations and their contracts are in include/rom.h.
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/rom.h"
#include "rom_internal.cuh"
#include "sm100_ptx.cuh"

namespace rom {

// One device status word per device (set by bounded waits that ran out).
__device__ int g_status_word;

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sm_count[kMaxDevices];
int* g_status_ptr[kMaxDevices];

int current_device() {
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return -1;
  return d;
}

// A buffer's bytes; a null one overlaps nothing.
struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int to_status(cudaError_t e) {
  if (e == cudaSuccess) return ROM_OK;
  if (e == cudaErrorInvalidValue) return ROM_ERR_UNSUPPORTED;
  return ROM_ERR_CUDA;
}

__global__ void debug_wait_kernel(uint64_t limit_ns, int* status) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  // Nothing ever arrives on `bar`: the wait must run out and report.
  if (threadIdx.x == 0) mbar_wait(&bar, 0, &abort_flag, status, limit_ns);
}

}  // namespace

int* status_ptr() {
  const int d = current_device();
  if (d < 0) return nullptr;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_status_ptr[d]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
    g_status_ptr[d] = static_cast<int*>(p);
  }
  return g_status_ptr[d];
}

int device_sm_count() {
  const int d = current_device();
  if (d < 0) return 1;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_sm_count[d] <= 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess || n <= 0)
      n = 1;
    g_sm_count[d] = n;
  }
  return g_sm_count[d];
}

}  // namespace rom

using rom::aligned16;
using rom::overlap;
using rom::Span;

extern "C" {

const char* rom_status_string(int status) {
  switch (status) {
    case ROM_OK:
      return "ROM_OK";
    case ROM_ERR_INVALID_ARG:
      return "ROM_ERR_INVALID_ARG";
    case ROM_ERR_UNSUPPORTED:
      return "ROM_ERR_UNSUPPORTED";
    case ROM_ERR_WORKSPACE:
      return "ROM_ERR_WORKSPACE";
    case ROM_ERR_CUDA:
      return "ROM_ERR_CUDA";
    case ROM_ERR_TIMEOUT:
      return "ROM_ERR_TIMEOUT";
    case ROM_ERR_ROUTING:
      return "ROM_ERR_ROUTING";
    default:
      return "ROM_ERR_UNKNOWN";
  }
}

int rom_version(void) { return 2; }

size_t rom_workspace_size(int64_t T, int E) {
  if (T <= 0 || E <= 0) return 0;
  return static_cast<size_t>(rom::num_chunks(T)) * static_cast<size_t>(E) * sizeof(int32_t);
}

int rom_route(const void* x, int dtype, int64_t T, int Dm, const float* w_r, const float* bias,
              int E, int k, int renorm, int32_t* topk_idx, float* topk_w, int32_t* counts,
              void* ws, size_t ws_bytes, void* stream) {
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (T < 0 || Dm <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E ||
      k > rom::kMaxTopK || (renorm != 0 && renorm != 1))
    return ROM_ERR_INVALID_ARG;
  if (T * k >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  const bool bf16 = dtype == ROM_BF16;
  if (Dm % (bf16 ? 8 : 4) != 0) return ROM_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T > 0) {
    if (!x || !w_r || !topk_idx || !topk_w) return ROM_ERR_INVALID_ARG;
    if (!aligned16(x)) return ROM_ERR_UNSUPPORTED;
    if (ws && ws_bytes < rom_workspace_size(T, E)) return ROM_ERR_WORKSPACE;
  }
  if (counts) {
    const cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * E, s);
    if (e != cudaSuccess) return ROM_ERR_CUDA;
  }
  if (T == 0) return ROM_OK;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_router(x, bf16, T, Dm, w_r, bias, E, k, renorm, topk_idx,
                                           topk_w, counts, static_cast<int32_t*>(ws), st, s));
}

int rom_dispatch(const void* x, int dtype, int64_t T, int Dm, int E, int k,
                 const int32_t* topk_idx, const void* ws, size_t ws_bytes, int32_t* offsets,
                 int32_t* sorted_slot, int32_t* slot_pos, void* x_sorted, void* stream) {
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (T < 0 || Dm <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E || k > rom::kMaxTopK)
    return ROM_ERR_INVALID_ARG;
  if (T * k >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  const bool bf16 = dtype == ROM_BF16;
  if (Dm % (bf16 ? 8 : 4) != 0) return ROM_ERR_UNSUPPORTED;
  if (!offsets) return ROM_ERR_INVALID_ARG;
  if (T > 0) {
    if (!x || !topk_idx || !sorted_slot || !slot_pos || !x_sorted) return ROM_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(x_sorted)) return ROM_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < rom_workspace_size(T, E)) return ROM_ERR_WORKSPACE;
  }
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_dispatch(x, bf16, T, Dm, E, k, topk_idx,
                                             static_cast<const int32_t*>(ws), offsets,
                                             sorted_slot, slot_pos, x_sorted, st,
                                             static_cast<cudaStream_t>(stream)));
}

int rom_expert_proj(int proj, int dtype, const void* a_sorted, int64_t R, int K, const void* w0,
                    const void* w1, int N, int E, int k, const int32_t* offsets,
                    const int32_t* sorted_slot, const float* topk_w, void* out, void* stream) {
  if (proj != ROM_PROJ_CONV_GATE && proj != ROM_PROJ_OUT && proj != ROM_PROJ_INPROJ &&
      proj != ROM_PROJ_SLOTS && proj != ROM_PROJ_CONV_GATE_SLOTS)
    return ROM_ERR_INVALID_ARG;
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (R < 0 || K <= 0 || N <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E ||
      k > rom::kMaxTopK || R % k != 0)
    return ROM_ERR_INVALID_ARG;
  if (R >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  const bool gate = proj == ROM_PROJ_CONV_GATE || proj == ROM_PROJ_CONV_GATE_SLOTS;
  const bool gate_slots = proj == ROM_PROJ_CONV_GATE_SLOTS || (gate && k > 1);
  const bool slots = proj == ROM_PROJ_SLOTS;
  // A dense projection (ROM_PROJ_SLOTS only): no routing arrays, one matrix.
  const bool dense = slots && !offsets && !sorted_slot;
  if (dense && E != 1) return ROM_ERR_INVALID_ARG;
  if ((!offsets && !dense) || !w0 || !out || (gate && !w1)) return ROM_ERR_INVALID_ARG;
  if (!gate && !dense && (!sorted_slot || (!slots && !topk_w))) return ROM_ERR_INVALID_ARG;
  if (gate_slots && !sorted_slot) return ROM_ERR_INVALID_ARG;
  if (R > 0 && !a_sorted) return ROM_ERR_INVALID_ARG;
  if (slots) w1 = nullptr;
  // ROM_PROJ_SLOTS is the slot-order float32 epilogue; r = 1 when topk_w is
  // NULL, and row p is slot p when sorted_slot is NULL.
  const int mode = gate    ? (gate_slots ? rom::kEpiGateSlots : rom::kEpiGateH)
                   : slots ? rom::kEpiScaleSlots
                           : (k == 1 ? rom::kEpiScaleToken : rom::kEpiScaleSlots);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == ROM_F32) {
    return rom::to_status(rom::launch_simt_grouped_gemm(
        mode, static_cast<const float*>(a_sorted), R, K, static_cast<const float*>(w0),
        static_cast<const float*>(w1), N, E, k, offsets, sorted_slot, topk_w,
        static_cast<float*>(out), s));
  }
  if (K % 8 != 0 || N % 128 != 0) return ROM_ERR_UNSUPPORTED;
  if (!aligned16(a_sorted) || !aligned16(w0) || (gate && !aligned16(w1)) || !aligned16(out))
    return ROM_ERR_UNSUPPORTED;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_tc_grouped_gemm(mode, a_sorted, R, K, w0, w1, N, E, k,
                                                    offsets, sorted_slot, topk_w, out, st, s));
}

int rom_expert_proj_dense(int proj, int dtype, const void* x, int64_t T, int K, const void* w,
                          int N, int E, int k, const int32_t* topk_idx, const float* topk_w,
                          void* out, void* stream) {
  const bool w_tiled = (proj & ROM_W_TILED) != 0;
  proj &= ~ROM_W_TILED;
  if (proj != ROM_PROJ_OUT && proj != ROM_PROJ_INPROJ) return ROM_ERR_INVALID_ARG;
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (T < 0 || K <= 0 || N <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E ||
      k > rom::kMaxTopK)
    return ROM_ERR_INVALID_ARG;
  if (dtype != ROM_BF16 || T > 64 || K % 8 != 0 || N % 128 != 0) return ROM_ERR_UNSUPPORTED;
  if (w_tiled && K % 64 != 0) return ROM_ERR_UNSUPPORTED;
  if (T == 0) return ROM_OK;
  if (!x || !w || !topk_idx || !topk_w || !out) return ROM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(out)) return ROM_ERR_UNSUPPORTED;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_tc_dense_small(
      k == 1 ? rom::kEpiScaleToken : rom::kEpiScaleSlots, x, T, K, w, N, E, k, topk_idx, topk_w,
      out, w_tiled, st, static_cast<cudaStream_t>(stream)));
}

int rom_pack_expert_weights(int dtype, const void* w, int E, int N, int K, void* w_tiled,
                            void* stream) {
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (E < 1 || N <= 0 || K <= 0) return ROM_ERR_INVALID_ARG;
  if (dtype != ROM_BF16 || N % 128 != 0 || K % 64 != 0) return ROM_ERR_UNSUPPORTED;
  if (!w || !w_tiled) return ROM_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(w_tiled)) return ROM_ERR_UNSUPPORTED;
  const uintptr_t a = reinterpret_cast<uintptr_t>(w), b = reinterpret_cast<uintptr_t>(w_tiled);
  const uintptr_t bytes = static_cast<uintptr_t>(E) * N * K * 2;
  if (a < b + bytes && b < a + bytes) return ROM_ERR_INVALID_ARG;  // overlapping
  return rom::to_status(rom::launch_pack_expert_weights(w, E, N, K, w_tiled,
                                                        static_cast<cudaStream_t>(stream)));
}

int rom_combine(int mode, int dtype, const void* in, int64_t T, int k, int N,
                const int32_t* slot_pos, void* out, void* stream) {
  if (mode != ROM_COMBINE_SUM && mode != ROM_COMBINE_GATE && mode != ROM_COMBINE_GATE_DENSE)
    return ROM_ERR_INVALID_ARG;
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (T < 0 || k < 1 || k > rom::kMaxTopK || N <= 0) return ROM_ERR_INVALID_ARG;
  if (N % 4 != 0) return ROM_ERR_UNSUPPORTED;
  if (T == 0) return ROM_OK;
  if (!in || !out) return ROM_ERR_INVALID_ARG;
  if (!aligned16(in) || !aligned16(out)) return ROM_ERR_UNSUPPORTED;
  return rom::to_status(rom::launch_combine(mode, dtype == ROM_BF16,
                                            static_cast<const float*>(in), T, k, N, slot_pos,
                                            out, static_cast<cudaStream_t>(stream)));
}

int rom_get_status(void* stream, int32_t* host_status) {
  if (!host_status) return ROM_ERR_INVALID_ARG;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return ROM_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, st, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return ROM_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(st, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
    return ROM_ERR_CUDA;
  *host_status = v;
  return ROM_OK;
}

int rom_bwd_gather(const void* dout, int64_t T, int k, int N, const int32_t* sorted_slot,
                   const float* topk_w, void* rdo_sorted, void* stream) {
  if (T < 0 || k < 1 || k > rom::kMaxTopK || N <= 0) return ROM_ERR_INVALID_ARG;
  if (N % 8 != 0 || T * k >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  if (T == 0) return ROM_OK;
  if (!dout || !sorted_slot || !topk_w || !rdo_sorted) return ROM_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(rdo_sorted)) return ROM_ERR_UNSUPPORTED;
  return rom::to_status(rom::launch_scale_gather(dout, T * k, k, N, sorted_slot, topk_w,
                                                 rdo_sorted, static_cast<cudaStream_t>(stream)));
}

int rom_bwd_dgrad_out(const void* rdo_sorted, int64_t R, int Dm, const void* w_out, int De, int E,
                      int k, const int32_t* offsets, const int32_t* sorted_slot,
                      const void* h_sorted, float* g_slots, float* dr_part, void* stream) {
  if (R < 0 || Dm <= 0 || De <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E ||
      k > rom::kMaxTopK || R % k != 0)
    return ROM_ERR_INVALID_ARG;
  if (Dm % 64 != 0 || De % 256 != 0 || R >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  if (!offsets || !w_out || !sorted_slot || !h_sorted || !g_slots || !dr_part ||
      (R > 0 && !rdo_sorted))
    return ROM_ERR_INVALID_ARG;
  if (!aligned16(rdo_sorted) || !aligned16(w_out) || !aligned16(h_sorted) || !aligned16(g_slots))
    return ROM_ERR_UNSUPPORTED;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_bwd_dgrad_out(rdo_sorted, R, Dm, w_out, De, E, k, offsets,
                                                  sorted_slot, h_sorted, g_slots, dr_part, st,
                                                  static_cast<cudaStream_t>(stream)));
}

int rom_bwd_gate(const float* uz, const float* g_slots, int64_t T, int k, int De,
                 const int32_t* slot_pos, void* dhz_sorted, void* stream) {
  if (T < 0 || k < 1 || k > rom::kMaxTopK || De <= 0) return ROM_ERR_INVALID_ARG;
  if (De % 4 != 0) return ROM_ERR_UNSUPPORTED;
  if (T == 0) return ROM_OK;
  if (!uz || !g_slots || !slot_pos || !dhz_sorted) return ROM_ERR_INVALID_ARG;
  if (!aligned16(uz) || !aligned16(g_slots) || !aligned16(dhz_sorted)) return ROM_ERR_UNSUPPORTED;
  return rom::to_status(rom::launch_gate_bwd(uz, g_slots, T, k, De, slot_pos, dhz_sorted,
                                             static_cast<cudaStream_t>(stream)));
}

int rom_bwd_dgrad_in(const void* dhz_sorted, int64_t R, int De, const void* w_in,
                     const void* w_g, int Dm, int E, int k, const int32_t* offsets,
                     const int32_t* sorted_slot, float* dx_slots, void* stream) {
  if (R < 0 || Dm <= 0 || De <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E ||
      k > rom::kMaxTopK || R % k != 0)
    return ROM_ERR_INVALID_ARG;
  if (De % 64 != 0 || Dm % 256 != 0 || R >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  if (!offsets || !w_in || !w_g || !sorted_slot || !dx_slots || (R > 0 && !dhz_sorted))
    return ROM_ERR_INVALID_ARG;
  if (!aligned16(dhz_sorted) || !aligned16(w_in) || !aligned16(w_g) || !aligned16(dx_slots))
    return ROM_ERR_UNSUPPORTED;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_bwd_dgrad_in(dhz_sorted, R, De, w_in, w_g, Dm, E, k, offsets,
                                                 sorted_slot, dx_slots, st,
                                                 static_cast<cudaStream_t>(stream)));
}

int rom_route_bwd(int64_t T, int k, int E, int Dm, int renorm, const int32_t* topk_idx,
                  const float* topk_w, const float* probs, const float* dr_part, int n_parts,
                  const float* dx_slots, const float* w_r, float* dlogits, void* dx,
                  void* stream) {
  if (T < 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E || k > rom::kMaxTopK || Dm <= 0 ||
      n_parts < 1 || (renorm != 0 && renorm != 1))
    return ROM_ERR_INVALID_ARG;
  if (Dm % 4 != 0) return ROM_ERR_UNSUPPORTED;
  if (T == 0) return ROM_OK;
  if (!topk_idx || !topk_w || !dr_part || !dx_slots || !w_r || !dx || (renorm == 0 && !probs))
    return ROM_ERR_INVALID_ARG;
  if (!aligned16(dx_slots) || !aligned16(w_r) || (reinterpret_cast<uintptr_t>(dx) & 7u))
    return ROM_ERR_UNSUPPORTED;
  return rom::to_status(rom::launch_route_bwd(T, k, E, Dm, topk_idx, topk_w,
                                              renorm ? nullptr : probs, dr_part, n_parts,
                                              dx_slots, w_r, dlogits, dx,
                                              static_cast<cudaStream_t>(stream)));
}

int rom_route_probs(const void* x, int dtype, int64_t T, int Dm, const float* w_r,
                    const float* bias, int E, float* probs, void* stream) {
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (T < 0 || Dm <= 0 || E < 1 || E > rom::kMaxExperts) return ROM_ERR_INVALID_ARG;
  if (T > 0 && (!x || !w_r || !probs)) return ROM_ERR_INVALID_ARG;
  return rom::to_status(rom::launch_route_probs(x, dtype == ROM_BF16, T, Dm, w_r, bias, E, probs,
                                                static_cast<cudaStream_t>(stream)));
}

int rom_bwd_wgrad(const void* a_sorted, int M, const void* b_sorted, int N, int64_t R, int E,
                  const int32_t* offsets, int m_split, float* out0, float* out1, void* stream) {
  if (M <= 0 || N <= 0 || R < 0 || E < 1 || E > rom::kMaxExperts || m_split < 0 || m_split > M)
    return ROM_ERR_INVALID_ARG;
  if (M % 128 != 0 || N % 256 != 0 || m_split % 128 != 0 || R >= (int64_t(1) << 31))
    return ROM_ERR_UNSUPPORTED;
  if (!a_sorted || !b_sorted || !offsets || !out0 || (m_split < M && !out1))
    return ROM_ERR_INVALID_ARG;
  if (!aligned16(a_sorted) || !aligned16(b_sorted) || !aligned16(out0) ||
      (out1 && !aligned16(out1)))
    return ROM_ERR_UNSUPPORTED;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_bwd_wgrad(a_sorted, M, b_sorted, N, R, E, offsets, m_split,
                                              out0, out1, st, static_cast<cudaStream_t>(stream)));
}

int rom_route_wgrad(const void* x, int dtype, int64_t T, int Dm, int E, const float* dlogits,
                    float* dw_r, float* dbias, void* stream) {
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (T < 0 || Dm <= 0 || E < 1 || E > rom::kMaxExperts) return ROM_ERR_INVALID_ARG;
  if (!dw_r || (T > 0 && (!x || !dlogits))) return ROM_ERR_INVALID_ARG;
  return rom::to_status(rom::launch_route_wgrad(x, dtype == ROM_BF16, T, Dm, E, dlogits, dw_r,
                                                dbias, static_cast<cudaStream_t>(stream)));
}

int rom_debug_wait_timeout(uint64_t limit_ns, void* stream) {
  if (limit_ns < 1000ull || limit_ns > 10000000000ull) return ROM_ERR_INVALID_ARG;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  rom::debug_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns, st);
  return rom::to_status(cudaGetLastError());
}

int rom_add_rmsnorm(const void* x, int dtype, const void* res, int res_dtype, int64_t T, int Dm,
                    const float* w, float eps, void* res_out, void* y, void* y8, float* y_scale,
                    float* rstd, void* stream) {
  if ((dtype != ROM_F32 && dtype != ROM_BF16) || (res_dtype != ROM_F32 && res_dtype != ROM_BF16))
    return ROM_ERR_INVALID_ARG;
  if (T < 0 || Dm <= 0 || !(eps > 0.f) || eps > 3.4e38f) return ROM_ERR_INVALID_ARG;
  if (!y8 != !y_scale) return ROM_ERR_INVALID_ARG;
  if (dtype == ROM_F32 && res_dtype != ROM_F32) return ROM_ERR_UNSUPPORTED;
  if (Dm % 8 != 0 || Dm > rom::kNormMaxCols || T >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  if (T == 0) return ROM_OK;
  if (!x || !w || (!res_out && !y && !y8 && !rstd)) return ROM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(res) || !aligned16(w) || !aligned16(res_out) || !aligned16(y) ||
      !aligned16(y8))
    return ROM_ERR_UNSUPPORTED;
  // outputs overlap nothing, but for res_out on res and y on x as a whole
  const size_t n = static_cast<size_t>(T) * Dm;
  const size_t xb = n * (dtype == ROM_BF16 ? 2 : 4), rb = n * (res_dtype == ROM_BF16 ? 2 : 4);
  const Span in[] = {{x, xb}, {res, rb}, {w, sizeof(float) * Dm}};
  const Span out[] = {{res_out, rb}, {y, xb}, {y8, n}, {y_scale, sizeof(float) * T},
                      {rstd, sizeof(float) * T}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 3; ++j) {
      const bool same = (i == 0 && j == 1 && res_out == res) || (i == 1 && j == 0 && y == x);
      if (!same && overlap(out[i], in[j])) return ROM_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return ROM_ERR_INVALID_ARG;
  }
  return rom::to_status(rom::launch_add_rmsnorm(x, dtype == ROM_BF16, res, res_dtype == ROM_BF16,
                                                T, Dm, w, eps, res_out, y, y8, y_scale, rstd,
                                                static_cast<cudaStream_t>(stream)));
}

size_t rom_add_rmsnorm_bwd_workspace_size(int64_t T, int Dm) {
  if (T <= 0 || Dm <= 0) return 0;
  const int64_t parts = T < rom::kNormBwdMaxParts ? T : rom::kNormBwdMaxParts;
  return static_cast<size_t>(parts) * static_cast<size_t>(Dm) * sizeof(float);
}

int rom_add_rmsnorm_bwd(const void* dy, int dtype, const void* dres_out, const void* res_out,
                        int res_dtype, int64_t T, int Dm, const float* w, const float* rstd,
                        void* dx, void* dres, float* dw, void* ws, size_t ws_bytes, void* stream) {
  if ((dtype != ROM_F32 && dtype != ROM_BF16) || (res_dtype != ROM_F32 && res_dtype != ROM_BF16))
    return ROM_ERR_INVALID_ARG;
  if (T < 0 || Dm <= 0) return ROM_ERR_INVALID_ARG;
  if (dtype == ROM_F32 && res_dtype != ROM_F32) return ROM_ERR_UNSUPPORTED;
  if (Dm % 8 != 0 || Dm > rom::kNormMaxCols || T >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dw && cudaMemsetAsync(dw, 0, sizeof(float) * Dm, s) != cudaSuccess) return ROM_ERR_CUDA;
    return ROM_OK;
  }
  if (!dy || !res_out || !w || !rstd || (!dx && !dres && !dw)) return ROM_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(dres_out) || !aligned16(res_out) || !aligned16(w) ||
      !aligned16(dx) || !aligned16(dres) || !aligned16(ws))
    return ROM_ERR_UNSUPPORTED;
  const size_t need = rom_add_rmsnorm_bwd_workspace_size(T, Dm);
  if (dw && (!ws || ws_bytes < need)) return ROM_ERR_WORKSPACE;
  const size_t n = static_cast<size_t>(T) * Dm;
  const size_t xb = n * (dtype == ROM_BF16 ? 2 : 4), rb = n * (res_dtype == ROM_BF16 ? 2 : 4);
  const Span in[] = {{dy, xb}, {dres_out, rb}, {res_out, rb}, {w, sizeof(float) * Dm},
                     {rstd, sizeof(float) * T}};
  const Span out[] = {{dx, xb}, {dres, rb}, {dw, sizeof(float) * Dm}, {dw ? ws : nullptr, need}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 5; ++j) {
      const bool same = i == 1 && j == 1 && dres == dres_out;
      if (!same && overlap(out[i], in[j])) return ROM_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return ROM_ERR_INVALID_ARG;
  }
  return rom::to_status(rom::launch_add_rmsnorm_bwd(dy, dtype == ROM_BF16, dres_out, res_out,
                                                    res_dtype == ROM_BF16, T, Dm, w, rstd, dx,
                                                    dres, dw, static_cast<float*>(ws), s));
}

int rom_quant_rows(const void* x, int dtype, int64_t rows, int K, void* q, float* scale,
                   void* stream) {
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (rows < 0 || K <= 0) return ROM_ERR_INVALID_ARG;
  if (K % 8 != 0 || K > rom::kNormMaxCols || rows >= (int64_t(1) << 31)) return ROM_ERR_UNSUPPORTED;
  if (rows == 0) return ROM_OK;
  if (!x || !q || !scale) return ROM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q)) return ROM_ERR_UNSUPPORTED;
  const size_t n = static_cast<size_t>(rows) * K;
  const Span xs = {x, n * (dtype == ROM_BF16 ? 2 : 4)}, qs = {q, n},
             ss = {scale, sizeof(float) * rows};
  if (overlap(xs, qs) || overlap(xs, ss) || overlap(qs, ss)) return ROM_ERR_INVALID_ARG;
  return rom::to_status(rom::launch_quant_rows(x, dtype == ROM_BF16, rows, K, q, scale,
                                               static_cast<cudaStream_t>(stream)));
}

int rom_dispatch_q8(const void* x8, const float* x_scale, int64_t T, int Dm, int E, int k,
                    const int32_t* topk_idx, const void* ws, size_t ws_bytes, int32_t* offsets,
                    int32_t* sorted_slot, int32_t* slot_pos, void* x8_sorted, float* scale_sorted,
                    void* stream) {
  if (T < 0 || Dm <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E || k > rom::kMaxTopK)
    return ROM_ERR_INVALID_ARG;
  if (T * k >= (int64_t(1) << 31) || Dm % 16 != 0) return ROM_ERR_UNSUPPORTED;
  if (!offsets) return ROM_ERR_INVALID_ARG;
  if (T > 0) {
    if (!x8 || !x_scale || !topk_idx || !sorted_slot || !slot_pos || !x8_sorted || !scale_sorted)
      return ROM_ERR_INVALID_ARG;
    if (!aligned16(x8) || !aligned16(x8_sorted)) return ROM_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < rom_workspace_size(T, E)) return ROM_ERR_WORKSPACE;
  }
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_dispatch_q8(x8, x_scale, T, Dm, E, k, topk_idx,
                                                static_cast<const int32_t*>(ws), offsets,
                                                sorted_slot, slot_pos, x8_sorted, scale_sorted, st,
                                                static_cast<cudaStream_t>(stream)));
}

int rom_expert_proj_q8(int proj, const void* a_sorted, const float* a_scale, int64_t R, int K,
                       const void* w0, const float* w0_scale, const void* w1,
                       const float* w1_scale, int N, int E, int k, const int32_t* offsets,
                       const int32_t* sorted_slot, const float* topk_w, void* out, void* stream) {
  if (proj != ROM_PROJ_CONV_GATE && proj != ROM_PROJ_OUT && proj != ROM_PROJ_INPROJ &&
      proj != ROM_PROJ_SLOTS && proj != ROM_PROJ_CONV_GATE_SLOTS)
    return ROM_ERR_INVALID_ARG;
  if (R < 0 || K <= 0 || N <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E ||
      k > rom::kMaxTopK || R % k != 0)
    return ROM_ERR_INVALID_ARG;
  if (R >= (int64_t(1) << 31) || K % 16 != 0 || N % 128 != 0) return ROM_ERR_UNSUPPORTED;
  if (R == 0) return ROM_OK;
  const bool gate = proj == ROM_PROJ_CONV_GATE || proj == ROM_PROJ_CONV_GATE_SLOTS;
  const bool gate_slots = proj == ROM_PROJ_CONV_GATE_SLOTS || (gate && k > 1);
  const bool slots = proj == ROM_PROJ_SLOTS;
  const bool dense = slots && !offsets && !sorted_slot;  // no routing arrays, one matrix
  if (dense && E != 1) return ROM_ERR_INVALID_ARG;
  if ((!offsets && !dense) || !w0 || !w0_scale || (gate && (!w1 || !w1_scale)))
    return ROM_ERR_INVALID_ARG;
  if (!gate && !dense && (!sorted_slot || (!slots && !topk_w))) return ROM_ERR_INVALID_ARG;
  if (gate_slots && !sorted_slot) return ROM_ERR_INVALID_ARG;
  if (!a_sorted || !a_scale || !out) return ROM_ERR_INVALID_ARG;
  if (!aligned16(a_sorted) || !aligned16(w0) || !aligned16(w0_scale) || !aligned16(out) ||
      (gate && (!aligned16(w1) || !aligned16(w1_scale))))
    return ROM_ERR_UNSUPPORTED;
  const int mode = gate    ? (gate_slots ? rom::kEpiGateSlots : rom::kEpiGateH)
                   : slots ? rom::kEpiScaleSlots
                           : (k == 1 ? rom::kEpiScaleToken : rom::kEpiScaleSlots);
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_tc_grouped_gemm_q8(
      mode, a_sorted, a_scale, R, K, w0, w0_scale, gate ? w1 : nullptr, gate ? w1_scale : nullptr,
      N, E, k, offsets, sorted_slot, topk_w, out, st, static_cast<cudaStream_t>(stream)));
}

size_t rom_w4_code_bytes(int E, int N, int K) {
  if (E < 1 || N <= 0 || K <= 0) return 0;
  return static_cast<size_t>(E) * ((static_cast<size_t>(N) + 15) / 16) *
         ((static_cast<size_t>(K) + 127) / 128) * 1024;
}

size_t rom_w4_scale_bytes(int E, int N, int K, int group) {
  if (group != 32 && group != 64 && group != 128) return 0;
  return rom_w4_code_bytes(E, N, K) / 1024 * 16 * (128 / group) * 2;
}

int rom_quant_expert_weights_w4(int dtype, const void* w, int E, int N, int K, int group, void* q,
                                void* s, void* stream) {
  if (dtype != ROM_F32 && dtype != ROM_BF16) return ROM_ERR_INVALID_ARG;
  if (E < 1 || N <= 0 || K <= 0 || (group != 32 && group != 64 && group != 128))
    return ROM_ERR_INVALID_ARG;
  const size_t qb = rom_w4_code_bytes(E, N, K), sb = rom_w4_scale_bytes(E, N, K, group);
  // one warp per 1 KB tile, eight to a block
  if (K % 8 != 0 || qb / 1024 >= (size_t(1) << 33) || N > (1 << 30) || K > (1 << 30))
    return ROM_ERR_UNSUPPORTED;
  if (!w || !q || !s) return ROM_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(q) || !aligned16(s)) return ROM_ERR_UNSUPPORTED;
  const Span wv = {w, static_cast<size_t>(E) * N * K * (dtype == ROM_BF16 ? 2 : 4)}, qv = {q, qb},
             sv = {s, sb};
  if (overlap(wv, qv) || overlap(wv, sv) || overlap(qv, sv)) return ROM_ERR_INVALID_ARG;
  return rom::to_status(rom::launch_quant_w4(w, dtype == ROM_BF16, E, N, K, group, q, s,
                                             static_cast<cudaStream_t>(stream)));
}

int rom_expert_proj_w4(int proj, const void* x, int64_t T, int K, const void* q0, const void* s0,
                       const void* q1, const void* s1, int N, int E, int k, int group,
                       const int32_t* topk_idx, const float* topk_w, void* out, void* stream) {
  const bool gate = proj == ROM_PROJ_CONV_GATE_SLOTS;
  const bool slots = proj == ROM_PROJ_SLOTS;
  if (!gate && !slots && proj != ROM_PROJ_OUT && proj != ROM_PROJ_INPROJ)
    return ROM_ERR_INVALID_ARG;
  if (T < 0 || K <= 0 || N <= 0 || E < 1 || E > rom::kMaxExperts || k < 1 || k > E ||
      k > rom::kMaxTopK || (group != 32 && group != 64 && group != 128))
    return ROM_ERR_INVALID_ARG;
  if (gate != (q1 != nullptr) || gate != (s1 != nullptr)) return ROM_ERR_INVALID_ARG;
  if (T > 64 || K % 8 != 0 || K > (1 << 24) || static_cast<int64_t>(E) * N > (1 << 30))
    return ROM_ERR_UNSUPPORTED;
  if (T == 0) return ROM_OK;
  if (!x || !q0 || !s0 || !topk_idx || !out || (!gate && !slots && !topk_w))
    return ROM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q0) || !aligned16(s0) || !aligned16(q1) || !aligned16(s1))
    return ROM_ERR_UNSUPPORTED;
  const bool to_token = !gate && !slots && k == 1;
  if ((reinterpret_cast<uintptr_t>(out) & (to_token ? 1u : 3u)) != 0) return ROM_ERR_UNSUPPORTED;
  int* st = rom::status_ptr();
  if (!st) return ROM_ERR_CUDA;
  return rom::to_status(rom::launch_w4_proj(x, static_cast<int>(T), K, q0, s0, q1, s1, N, E, k,
                                            group, topk_idx, gate ? nullptr : topk_w, out,
                                            to_token, st, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
