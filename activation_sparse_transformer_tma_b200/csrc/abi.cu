// abi.cu -- extern "C" entry points of libtwell.so: argument validation
// (before any launch) and dispatch to the kernels.  The library never
// allocates device memory and never synchronises the caller's stream.
#include <algorithm>
#include <cfloat>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "tw_internal.h"

namespace tw {

int num_sms() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v <= 0) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
      v = 1;
    cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

cudaError_t set_smem_limit(const void* func, int bytes) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, int> done;  // (kernel, device) -> bytes set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  auto it = done.find({func, dev});
  if (it != done.end() && it->second >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[{func, dev}] = bytes;
  return e;
}

namespace {
std::atomic<unsigned long long> g_withheld_gate_wait{0};
std::atomic<unsigned long long> g_withheld_ffn_wait{0};
}  // namespace

unsigned long long take_withheld_gate_wait() { return g_withheld_gate_wait.exchange(0); }
unsigned long long take_withheld_ffn_wait() { return g_withheld_ffn_wait.exchange(0); }

}  // namespace tw

namespace {

constexpr int kTileW = 128;    // the tile width of the dense comparators' F tiles
constexpr int kMaxRowD = 2048;

// TwELL tile widths: 64, 128 (the default) or 256 (tile-local indices are
// uint8).  Any capacity C up to the tile width.
bool tile_width_ok(int W) { return W == 64 || W == 128 || W == 256; }

}  // namespace

namespace tw {

// Row width d: a multiple of 8, at most 2048 for bf16 rows and 1024 for fp32
// rows (the gather engine keeps one token's row slices and its fp32 output
// slices in the registers of one team of warps).
bool row_d_ok(int d, tw_dtype t) {
  return d % 8 == 0 && d <= (t == TW_BF16 ? kMaxRowD : kMaxRowD / 2);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(tw_dtype t) { return t == TW_F32 || t == TW_BF16; }

// Shared checks of a TwELL descriptor.
tw_status check_twell(const tw_twell* g) {
  if (!g) return TW_ERR_INVALID_ARG;
  if (g->T < 0 || g->F <= 0 || g->C < 0 || g->spill_cap < 0 || !dtype_ok(g->dtype))
    return TW_ERR_INVALID_ARG;
  if (!tile_width_ok(g->W) || g->F % g->W != 0 || g->C > g->W) return TW_ERR_UNSUPPORTED;
  if (g->F > 65536) return TW_ERR_UNSUPPORTED;
  // arrays sized by T may be NULL for an empty batch
  if (!g->spill_n || (g->T > 0 && (!g->cnt || !g->spill_ref))) return TW_ERR_INVALID_ARG;
  if (g->T > 0 && g->C > 0 && (!g->val || !g->idx)) return TW_ERR_INVALID_ARG;
  if (g->spill_cap > 0 && (!g->spill_tk || !g->spill_val)) return TW_ERR_INVALID_ARG;
  if ((g->val && !aligned16(g->val)) || (g->idx && !aligned16(g->idx)) ||
      (g->spill_val && !aligned16(g->spill_val)))
    return TW_ERR_ALIGNMENT;
  return TW_OK;
}

}  // namespace tw

namespace {

using tw::aligned16;
using tw::check_twell;
using tw::dtype_ok;
using tw::row_d_ok;

tw_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TW_OK : TW_ERR_CUDA; }

tw_status check_hybrid(const tw_hybrid* h) {
  if (!h) return TW_ERR_INVALID_ARG;
  if (h->T < 0 || h->F <= 0 || h->C_h < 0 || h->C_h > h->F || h->backup_cap < 0 ||
      !dtype_ok(h->dtype))
    return TW_ERR_INVALID_ARG;
  // unit histograms live in shared memory; dense rows are read 16 bytes at a time
  if (h->F > 51200 || h->F % 8 != 0) return TW_ERR_UNSUPPORTED;
  if ((size_t)h->T * (size_t)h->C_h + (size_t)h->backup_cap * (size_t)h->F > 0x7FFFFFFFull)
    return TW_ERR_UNSUPPORTED;  // entry numbers are int32
  // arrays sized by T may be NULL for an empty batch
  if (!h->n_backup || (h->T > 0 && (!h->row_nnz || !h->row_slot))) return TW_ERR_INVALID_ARG;
  if (h->T > 0 && h->C_h > 0 && (!h->ell_g || !h->ell_idx)) return TW_ERR_INVALID_ARG;
  if (h->backup_cap > 0 && (!h->backup_rows || !h->backup_g)) return TW_ERR_INVALID_ARG;
  return TW_OK;
}

// One array of a call.  `over`: inputs whose whole array an output may take.
struct Span {
  const void* at;
  size_t bytes;
  bool written;
  const void* over[2];
};

// Whether no written array overlaps another one, but for the allowed whole arrays.
template <size_t N>
bool spans_apart(const Span (&spans)[N]) {
  for (size_t i = 0; i < N; ++i) {
    const Span& w = spans[i];
    if (!w.written || !w.at || w.bytes == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(w.at);
    for (size_t j = 0; j < N; ++j) {
      const Span& o = spans[j];
      if (j == i || !o.at || o.bytes == 0) continue;
      const uintptr_t b = reinterpret_cast<uintptr_t>(o.at);
      if (a >= b + o.bytes || b >= a + w.bytes) continue;
      if (!o.written && a == b && w.bytes == o.bytes && (o.at == w.over[0] || o.at == w.over[1]))
        continue;
      return false;
    }
  }
  return true;
}

size_t bytes_of(tw_dtype t) { return t == TW_BF16 ? 2 : 4; }

}  // namespace

extern "C" {

tw_status tw_measure_row_gather(const void* mat, int32_t rows, int32_t d, int64_t n_gathers,
                                uint32_t seed, uint32_t* checksum, cudaStream_t stream) {
  if (rows < 1 || d < 8 || d > 2048 || d % 8 != 0 || n_gathers < 0 || !mat || !checksum)
    return TW_ERR_INVALID_ARG;
  if (!aligned16(mat)) return TW_ERR_ALIGNMENT;
  if (n_gathers == 0) return TW_OK;
  return from_cuda(
      tw::launch_row_gather(mat, rows, d, (long long)n_gathers, seed, checksum, stream));
}

tw_status tw_measure_stream_read(const void* buf, int64_t bytes, uint32_t* checksum,
                                 cudaStream_t stream) {
  if (bytes < 0 || bytes % 16 != 0 || !buf || !checksum) return TW_ERR_INVALID_ARG;
  if (!aligned16(buf)) return TW_ERR_ALIGNMENT;
  if (bytes == 0) return TW_OK;
  return from_cuda(tw::launch_stream_read(buf, (long long)bytes, checksum, stream));
}

const char* tw_status_string(tw_status s) {
  switch (s) {
    case TW_OK: return "TW_OK";
    case TW_ERR_INVALID_ARG: return "TW_ERR_INVALID_ARG";
    case TW_ERR_UNSUPPORTED: return "TW_ERR_UNSUPPORTED";
    case TW_ERR_ALIGNMENT: return "TW_ERR_ALIGNMENT";
    case TW_ERR_CUDA: return "TW_ERR_CUDA";
    case TW_ERR_SPILL_CAPACITY: return "TW_ERR_SPILL_CAPACITY";
    case TW_ERR_BACKUP_CAPACITY: return "TW_ERR_BACKUP_CAPACITY";
    case TW_ERR_TIMEOUT: return "TW_ERR_TIMEOUT";
    case TW_ERR_WORKSPACE: return "TW_ERR_WORKSPACE";
  }
  return "TW_UNKNOWN_STATUS";
}

int32_t twell_version(void) { return 200; }

void tw_test_withhold_next_gate_loads(uint64_t wait_limit_ns) {
  tw::g_withheld_gate_wait.store(wait_limit_ns > 0 ? wait_limit_ns : 1);
}

void tw_test_withhold_next_gated_ffn_loads(uint64_t wait_limit_ns) {
  tw::g_withheld_ffn_wait.store(wait_limit_ns > 0 ? wait_limit_ns : 1);
}

tw_status twell_gate_gemm(const void* x, const void* Wg_t, int32_t T, int32_t d, int32_t F,
                          tw_dtype dtype, const tw_twell* out, void* g_dense_dump,
                          int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_twell(out);
  if (st != TW_OK) return st;
  if ((T > 0 && !x) || !Wg_t) return TW_ERR_INVALID_ARG;
  if (T < 0 || d <= 0 || F <= 0 || out->T != T || out->F != F || out->dtype != dtype)
    return TW_ERR_INVALID_ARG;
  if (d % 8 != 0) return TW_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(Wg_t) || (g_dense_dump && !aligned16(g_dense_dump)))
    return TW_ERR_ALIGNMENT;
  if (T == 0) return from_cuda(cudaMemsetAsync(out->spill_n, 0, sizeof(int32_t), stream));
  if (dtype == TW_BF16) {
    if (d < 64) return TW_ERR_UNSUPPORTED;
    if (T <= tw::kFewMaxT && out->W == 128)
      return from_cuda(tw::launch_gate_twell_few(x, Wg_t, T, d, F, *out, g_dense_dump,
                                                 dev_status, stream));
    return from_cuda(tw::launch_gate_twell_tc(x, Wg_t, T, d, F, *out, g_dense_dump, dev_status,
                                              stream));
  }
  return from_cuda(tw::launch_gate_twell_f32(static_cast<const float*>(x),
                                             static_cast<const float*>(Wg_t), T, d, F, *out,
                                             static_cast<float*>(g_dense_dump), dev_status,
                                             stream));
}

size_t twell_fused_updown_workspace_size(int32_t T, int32_t d) {
  if (T < 0 || d <= 0) return 0;
  return tw::fused_ws_bytes(T, d);
}

tw_status twell_fused_updown(const void* x, const tw_twell* g, const void* Wu_t, const void* Wd,
                             int32_t d, void* y, tw_dtype y_dtype, void* ws, size_t ws_bytes,
                             int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_twell(g);
  if (st != TW_OK) return st;
  const bool any = g->T > 0;  // with no tokens x, y and ws are not touched
  if ((any && (!x || !y || !ws)) || !Wu_t || !Wd || !dtype_ok(y_dtype)) return TW_ERR_INVALID_ARG;
  if (d <= 0) return TW_ERR_INVALID_ARG;
  if (!row_d_ok(d, g->dtype)) return TW_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(Wu_t) || !aligned16(Wd) || !aligned16(y) || !aligned16(ws))
    return TW_ERR_ALIGNMENT;
  if (!any) return TW_OK;
  if (ws_bytes < tw::fused_ws_bytes(g->T, d)) return TW_ERR_WORKSPACE;
  return from_cuda(
      tw::launch_fused_updown(x, *g, Wu_t, Wd, d, y, y_dtype, ws, dev_status, stream));
}

tw_status twell_to_hybrid(const tw_twell* g, const tw_hybrid* out, int32_t* dev_status,
                          cudaStream_t stream) {
  tw_status st = check_twell(g);
  if (st != TW_OK) return st;
  st = check_hybrid(out);
  if (st != TW_OK) return st;
  if (out->T != g->T || out->F != g->F || out->dtype != g->dtype) return TW_ERR_INVALID_ARG;
  if (g->T == 0) return from_cuda(cudaMemsetAsync(out->n_backup, 0, sizeof(int32_t), stream));
  return from_cuda(tw::launch_twell_to_hybrid(*g, *out, dev_status, stream));
}

size_t hybrid_ffn_forward_workspace_size(int32_t T, int32_t d) {
  if (T < 0 || d <= 0) return 0;
  return tw::hybrid_forward_ws_bytes(T, d);
}

tw_status hybrid_ffn_forward(const void* x, const tw_hybrid* gu, const void* Wu_t,
                             const void* Wd, int32_t d, void* y, tw_dtype y_dtype, void* ws,
                             size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_hybrid(gu);
  if (st != TW_OK) return st;
  const bool any = gu->T > 0;  // with no tokens x, y, ws and ell_u are not touched
  if ((any && (!x || !y || !ws)) || !Wu_t || !Wd || !dtype_ok(y_dtype)) return TW_ERR_INVALID_ARG;
  if ((any && gu->C_h > 0 && !gu->ell_u) || (gu->backup_cap > 0 && !gu->backup_u))
    return TW_ERR_INVALID_ARG;
  if (d <= 0) return TW_ERR_INVALID_ARG;
  if (!row_d_ok(d, gu->dtype)) return TW_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(Wu_t) || !aligned16(Wd) || !aligned16(y) || !aligned16(ws))
    return TW_ERR_ALIGNMENT;
  if (any && ws_bytes < tw::hybrid_forward_ws_bytes(gu->T, d)) return TW_ERR_WORKSPACE;
  return from_cuda(
      tw::launch_hybrid_forward(x, *gu, Wu_t, Wd, d, y, y_dtype, ws, dev_status, stream));
}

size_t hybrid_ffn_backward_workspace_size(int32_t T, int32_t d, int32_t F, int32_t C_h,
                                          int32_t backup_cap) {
  if (T < 0 || F <= 0 || C_h < 0 || backup_cap < 0) return 0;
  return tw::hybrid_backward_ws_bytes(T, d, F, C_h, backup_cap);
}

tw_status hybrid_ffn_backward(const void* x, const void* dy, const tw_hybrid* gu,
                              const void* Wg_t, const void* Wu_t, const void* Wd, int32_t d,
                              float l1_lambda, void* dx, tw_dtype dx_dtype, float* dWg_t,
                              float* dWu_t, float* dWd, void* ws, size_t ws_bytes,
                              int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_hybrid(gu);
  if (st != TW_OK) return st;
  const bool any = gu->T > 0;  // with no tokens only the weight gradients are written
  if ((any && (!x || !dy || !dx || !ws)) || !Wg_t || !Wu_t || !Wd || !dWg_t || !dWu_t || !dWd ||
      !dtype_ok(dx_dtype))
    return TW_ERR_INVALID_ARG;
  if ((any && gu->C_h > 0 && !gu->ell_u) || (gu->backup_cap > 0 && !gu->backup_u))
    return TW_ERR_INVALID_ARG;
  if (d <= 0) return TW_ERR_INVALID_ARG;
  if (!row_d_ok(d, gu->dtype)) return TW_ERR_UNSUPPORTED;
  const void* ptrs[] = {x, dy, Wg_t, Wu_t, Wd, dx, dWg_t, dWu_t, dWd, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if (any && ws_bytes < tw::hybrid_backward_ws_bytes(gu->T, d, gu->F, gu->C_h, gu->backup_cap))
    return TW_ERR_WORKSPACE;
  return from_cuda(tw::launch_hybrid_backward(x, dy, *gu, Wg_t, Wu_t, Wd, d, l1_lambda, dx,
                                              dx_dtype, dWg_t, dWu_t, dWd, ws, ws_bytes,
                                              dev_status, stream));
}

tw_status dense_ffn_forward(const void* x, const void* Wg_t, const void* Wu_t,
                            const void* Wd_dense, int32_t T, int32_t d, int32_t F, void* h_ws,
                            void* y, int32_t* dev_status, cudaStream_t stream) {
  if (!x || !Wg_t || !Wu_t || !Wd_dense || !h_ws || !y) return TW_ERR_INVALID_ARG;
  if (T < 0 || d <= 0 || F <= 0) return TW_ERR_INVALID_ARG;
  if (d % 32 != 0 || d < 64 || F % kTileW != 0) return TW_ERR_UNSUPPORTED;
  const void* ptrs[] = {x, Wg_t, Wu_t, Wd_dense, h_ws, y};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if (T == 0) return TW_OK;
  cudaError_t e = tw::launch_dense_gateup_tc(x, Wg_t, Wu_t, T, d, F, h_ws, dev_status, stream);
  if (e != cudaSuccess) return TW_ERR_CUDA;
  return from_cuda(tw::launch_dense_down_tc(h_ws, Wd_dense, T, d, F, y, dev_status, stream));
}

size_t twell_ffn_small_batch_workspace_size(int32_t T, int32_t d, int32_t F) {
  if (T < 0 || d <= 0 || F <= 0) return 0;
  return tw::decode_ws_bytes(T, d, F);
}

tw_status twell_ffn_small_batch(const void* x, const void* Wg_t, const void* Wu_t, const void* Wd,
                                int32_t T, int32_t d, int32_t F, const tw_twell* g,
                                void* g_dense_dump, void* y, tw_dtype y_dtype, void* ws,
                                size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_twell(g);
  if (st != TW_OK) return st;
  if (g->T != T || g->F != F || T < 0 || d <= 0) return TW_ERR_INVALID_ARG;
  if ((T > 0 && (!x || !y || !ws)) || !Wg_t || !Wu_t || !Wd || !dtype_ok(y_dtype))
    return TW_ERR_INVALID_ARG;
  if (g->dtype != TW_BF16 || g->W != 128 || T > tw::kDecodeStepMaxT || d % 8 != 0 || d < 64 ||
      d > kMaxRowD)
    return TW_ERR_UNSUPPORTED;
  const void* ptrs[] = {x, Wg_t, Wu_t, Wd, y, ws, g_dense_dump};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if (T == 0) return from_cuda(cudaMemsetAsync(g->spill_n, 0, sizeof(int32_t), stream));
  if (ws_bytes < tw::decode_ws_bytes(T, d, F)) return TW_ERR_WORKSPACE;
  return from_cuda(tw::launch_decode_step(x, Wg_t, Wu_t, Wd, T, d, F, *g, g_dense_dump, y,
                                          y_dtype, ws, dev_status, stream));
}

static size_t gated_part(int32_t T, int32_t F) {
  return ((size_t)T * (size_t)F * 2 + 255) & ~size_t(255);
}

size_t gated_ffn_workspace_size(int32_t T, int32_t d, int32_t F) {
  if (T < 0 || d <= 0 || F <= 0) return 0;
  return gated_part(T, F) + tw::gated_forward_split_bytes(T, d, F);
}

size_t gated_ffn_backward_workspace_size(int32_t T, int32_t d, int32_t F) {
  if (T < 0 || d <= 0 || F <= 0) return 0;
  return 3 * gated_part(T, F) + tw::gated_backward_split_bytes(T, d, F);
}

static tw_status check_gated(int32_t T, int32_t d, int32_t F, tw_act act) {
  if (T < 0 || d <= 0 || F <= 0 || (int)act < TW_ACT_RELU || (int)act > TW_ACT_GELU_TANH)
    return TW_ERR_INVALID_ARG;
  if (d % 8 != 0 || F % 8 != 0 || d < 64 || F < 64) return TW_ERR_UNSUPPORTED;
  return TW_OK;
}

tw_status gated_ffn_forward(const void* x, const void* Wg_t, const void* Wu_t, const void* Wd,
                            int32_t T, int32_t d, int32_t F, tw_act act, void* z_save,
                            void* u_save, void* y, tw_dtype y_dtype, void* ws, size_t ws_bytes,
                            int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_gated(T, d, F, act);
  if (st != TW_OK) return st;
  if ((T > 0 && (!x || !y || !ws)) || !Wg_t || !Wu_t || !Wd || !dtype_ok(y_dtype) ||
      (z_save != nullptr) != (u_save != nullptr))
    return TW_ERR_INVALID_ARG;
  const void* ptrs[] = {x, Wg_t, Wu_t, Wd, z_save, u_save, y, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if (T == 0) return TW_OK;
  const size_t need = gated_ffn_workspace_size(T, d, F);
  if (ws_bytes < need) return TW_ERR_WORKSPACE;
  const size_t rows = (size_t)T * d, acts = (size_t)T * F * 2, w = (size_t)F * d * 2;
  const Span spans[] = {{x, rows * 2, false, {}},    {Wg_t, w, false, {}},
                        {Wu_t, w, false, {}},        {Wd, w, false, {}},
                        {z_save, acts, true, {}},    {u_save, acts, true, {}},
                        {y, rows * bytes_of(y_dtype), true, {}}, {ws, need, true, {}}};
  if (!spans_apart(spans)) return TW_ERR_INVALID_ARG;
  return from_cuda(tw::launch_gated_forward(x, Wg_t, Wu_t, Wd, T, d, F, act,
                                            static_cast<uint16_t*>(ws),
                                            static_cast<uint16_t*>(z_save),
                                            static_cast<uint16_t*>(u_save), y, y_dtype,
                                            static_cast<char*>(ws) + gated_part(T, F), dev_status,
                                            stream));
}

tw_status gated_ffn_backward(const void* x, const void* dy, const void* Wg_t, const void* Wu_t,
                             const void* Wd, int32_t T, int32_t d, int32_t F, tw_act act,
                             const void* z_save, const void* u_save, void* dx, tw_dtype dx_dtype,
                             void* dWg_t, void* dWu_t, void* dWd, tw_dtype dw_dtype, void* ws,
                             size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_gated(T, d, F, act);
  if (st != TW_OK) return st;
  if ((T > 0 && (!x || !dy || !z_save || !u_save || !dx || !ws)) || !Wg_t || !Wu_t || !Wd ||
      !dWg_t || !dWu_t || !dWd || !dtype_ok(dx_dtype) || !dtype_ok(dw_dtype))
    return TW_ERR_INVALID_ARG;
  const void* ptrs[] = {x, dy, Wg_t, Wu_t, Wd, z_save, u_save, dx, dWg_t, dWu_t, dWd, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  const size_t need = gated_ffn_backward_workspace_size(T, d, F);
  if (T > 0 && ws_bytes < need) return TW_ERR_WORKSPACE;
  const size_t rows = (size_t)T * d, acts = (size_t)T * F * 2, w = (size_t)F * d;
  const size_t dw = w * bytes_of(dw_dtype);
  const Span spans[] = {{x, rows * 2, false, {}},  {dy, rows * 2, false, {}},
                        {Wg_t, w * 2, false, {}},  {Wu_t, w * 2, false, {}},
                        {Wd, w * 2, false, {}},    {z_save, acts, false, {}},
                        {u_save, acts, false, {}}, {dx, rows * bytes_of(dx_dtype), true, {}},
                        {dWg_t, dw, true, {}},     {dWu_t, dw, true, {}},
                        {dWd, dw, true, {}},       {T > 0 ? ws : nullptr, need, true, {}}};
  if (!spans_apart(spans)) return TW_ERR_INVALID_ARG;
  if (T == 0) {  // no tokens: zero weight gradients
    const size_t bytes = dw;
    void* grads[] = {dWg_t, dWu_t, dWd};
    for (void* g : grads) {
      cudaError_t e = cudaMemsetAsync(g, 0, bytes, stream);
      if (e != cudaSuccess) return from_cuda(e);
    }
    return TW_OK;
  }
  uint16_t* base = static_cast<uint16_t*>(ws);
  const size_t part = gated_part(T, F) / 2;
  return from_cuda(tw::launch_gated_backward(
      x, dy, Wg_t, Wu_t, Wd, T, d, F, act, static_cast<const uint16_t*>(z_save),
      static_cast<const uint16_t*>(u_save), base, base + part, base + 2 * part, dx, dx_dtype, dWg_t,
      dWu_t, dWd, dw_dtype, base + 3 * part, dev_status, stream));
}

static tw_status check_norm_block(const tw_norm_block* b, bool has_y) {
  if (!b) return TW_ERR_INVALID_ARG;
  if (b->T < 0 || b->d <= 0 || !dtype_ok(b->y_dtype) || !dtype_ok(b->r_dtype) ||
      !dtype_ok(b->n_dtype) || !dtype_ok(b->w_dtype))
    return TW_ERR_INVALID_ARG;
  if (!(b->eps >= 0.f) || !std::isfinite(b->eps) || !std::isfinite(b->res_scale) ||
      !std::isfinite(b->block_scale))
    return TW_ERR_INVALID_ARG;
  if (b->d % 8 != 0 || b->d > tw::kNormMaxD) return TW_ERR_UNSUPPORTED;
  if (b->gate && b->gate_group < 1) return TW_ERR_INVALID_ARG;
  if (!has_y && (b->w_post || b->gate || !b->w_pre)) return TW_ERR_INVALID_ARG;
  if (!aligned16(b->w_post) || !aligned16(b->gate) || !aligned16(b->w_pre))
    return TW_ERR_ALIGNMENT;
  return TW_OK;
}

tw_status norm_residual_forward(const tw_norm_block* b, const void* y, const void* r, void* r_out,
                                void* n_out, float* rstd_post, float* rstd_pre,
                                cudaStream_t stream) {
  // with no tokens the arrays sized by T may all be NULL, y among them
  const bool any = b && b->T > 0;
  tw_status st = check_norm_block(b, !any || y);
  if (st != TW_OK) return st;
  const void* ptrs[] = {y, r, r_out, n_out, rstd_post, rstd_pre};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if (!any) return TW_OK;
  if (!r || (y != nullptr) != (r_out != nullptr)) return TW_ERR_INVALID_ARG;
  if ((b->w_pre != nullptr) != (n_out != nullptr) || (rstd_pre && !b->w_pre) ||
      (rstd_post && !b->w_post))
    return TW_ERR_INVALID_ARG;
  const size_t e = (size_t)b->T * b->d, d = (size_t)b->d * bytes_of(b->w_dtype), f = (size_t)b->T * 4;
  const size_t groups = b->gate ? ((size_t)b->T + b->gate_group - 1) / b->gate_group : 0;
  const bool yn = b->n_dtype == b->y_dtype, rn = b->n_dtype == b->r_dtype;
  const Span spans[] = {{y, e * bytes_of(b->y_dtype), false, {}},
                        {r, e * bytes_of(b->r_dtype), false, {}},
                        {b->w_post, d, false, {}},
                        {b->gate, groups * d, false, {}},
                        {b->w_pre, d, false, {}},
                        {r_out, e * bytes_of(b->r_dtype), true,
                         {r, b->y_dtype == b->r_dtype ? y : nullptr}},
                        {n_out, e * bytes_of(b->n_dtype), true, {yn ? y : nullptr, rn ? r : nullptr}},
                        {rstd_post, f, true, {}},
                        {rstd_pre, f, true, {}}};
  if (!spans_apart(spans)) return TW_ERR_INVALID_ARG;
  return from_cuda(
      tw::launch_norm_forward(*b, y, r, r_out, n_out, rstd_post, rstd_pre, stream));
}

size_t norm_residual_backward_workspace_size(int32_t T, int32_t d, int32_t gate_group) {
  // no tokens: nothing is summed; widths that the call refuses
  if (T <= 0 || d <= 0 || d % 8 != 0 || d > tw::kNormMaxD || gate_group < 0) return 0;
  return tw::norm_backward_ws_bytes(T, d, gate_group);
}

tw_status norm_residual_backward(const tw_norm_block* b, const void* dn, const void* dr_out,
                                 const void* y, const void* r_out, const float* rstd_post,
                                 const float* rstd_pre, void* dy, void* dr, float* dw_post,
                                 float* dgate, float* dw_pre, void* ws, size_t ws_bytes,
                                 cudaStream_t stream) {
  const bool any = b && b->T > 0;
  tw_status st = check_norm_block(b, !any || y);
  if (st != TW_OK) return st;
  const void* ptrs[] = {dn, dr_out, y, r_out, rstd_post, rstd_pre, dy, dr, dw_post, dgate, dw_pre,
                        ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if ((b->w_pre != nullptr) != (dw_pre != nullptr) || (b->w_post != nullptr) != (dw_post != nullptr))
    return TW_ERR_INVALID_ARG;
  if (!any) {  // no tokens: zero weight gradients, and no gate rows
    const size_t bytes = sizeof(float) * (size_t)b->d;
    cudaError_t e = dw_pre ? cudaMemsetAsync(dw_pre, 0, bytes, stream) : cudaSuccess;
    if (e == cudaSuccess && dw_post) e = cudaMemsetAsync(dw_post, 0, bytes, stream);
    return from_cuda(e);
  }
  if (!dr || (!dn && !dr_out) || (b->w_pre != nullptr) != (dn != nullptr)) return TW_ERR_INVALID_ARG;
  if ((y != nullptr) != (dy != nullptr) || (b->gate != nullptr) != (dgate != nullptr))
    return TW_ERR_INVALID_ARG;
  if ((b->w_pre != nullptr) != (rstd_pre != nullptr) ||
      (b->w_post != nullptr) != (rstd_post != nullptr) || (b->w_pre && !r_out))
    return TW_ERR_INVALID_ARG;
  if (!ws) return TW_ERR_INVALID_ARG;
  const size_t need = tw::norm_backward_ws_bytes(b->T, b->d, b->gate ? b->gate_group : 0);
  if (ws_bytes < need) return TW_ERR_WORKSPACE;
  const size_t e = (size_t)b->T * b->d, d = (size_t)b->d * bytes_of(b->w_dtype), f = (size_t)b->T * 4;
  const size_t groups = b->gate ? ((size_t)b->T + b->gate_group - 1) / b->gate_group : 0;
  const size_t er = e * bytes_of(b->r_dtype), ey = e * bytes_of(b->y_dtype), d4 = (size_t)b->d * 4;
  const Span spans[] = {{dn, e * bytes_of(b->n_dtype), false, {}},
                        {dr_out, er, false, {}},
                        {y, ey, false, {}},
                        {b->w_pre ? r_out : nullptr, er, false, {}},
                        {b->w_post, d, false, {}},
                        {b->gate, groups * d, false, {}},
                        {b->w_pre, d, false, {}},
                        {rstd_post, f, false, {}},
                        {rstd_pre, f, false, {}},
                        {dy, ey, true, {y, b->n_dtype == b->y_dtype ? dn : nullptr}},
                        {dr, er, true, {dr_out, nullptr}},
                        {dw_post, d4, true, {}},
                        {dgate, groups * d4, true, {}},
                        {dw_pre, d4, true, {}},
                        {ws, need, true, {}}};
  if (!spans_apart(spans)) return TW_ERR_INVALID_ARG;
  return from_cuda(tw::launch_norm_backward(*b, dn, dr_out, y, r_out, rstd_post, rstd_pre, dy, dr,
                                            dw_post, dgate, dw_pre, ws, stream));
}

// One array of an optimiser step, for the check that written arrays are apart.
struct AdamwRange {
  uintptr_t first, last;
  bool written;
};

static tw_status check_adamw_tensor(const tw_adamw_tensor& t, std::vector<AdamwRange>* ranges) {
  if (t.n < 0 || !dtype_ok(t.p_dtype) || !dtype_ok(t.g_dtype) ||
      !(t.weight_decay >= 0.0 && std::isfinite(t.weight_decay)))
    return TW_ERR_INVALID_ARG;
  if (t.state_bits != 8 && t.state_bits != 32) return TW_ERR_UNSUPPORTED;
  if (t.n > (int64_t(1) << 40)) return TW_ERR_UNSUPPORTED;
  const bool small = t.state_bits == 8;
  if (t.n == 0) return TW_OK;
  if (!t.p || !t.g || !t.m || !t.v) return TW_ERR_INVALID_ARG;
  if (t.master && t.p_dtype != TW_BF16) return TW_ERR_INVALID_ARG;
  if (small != (t.m_scale != nullptr) || small != (t.v_scale != nullptr)) return TW_ERR_INVALID_ARG;
  if ((t.m_values != nullptr) != (t.v_values != nullptr)) return TW_ERR_INVALID_ARG;
  if (t.m_values && (!small || !dtype_ok(t.values_dtype))) return TW_ERR_INVALID_ARG;
  const size_t n = (size_t)t.n, blocks = (n + TW_ADAMW_BLOCK - 1) / TW_ADAMW_BLOCK;
  const size_t pb = t.p_dtype == TW_BF16 ? 2 : 4, gb = t.g_dtype == TW_BF16 ? 2 : 4;
  const size_t sb = small ? 1 : 4, vb = t.values_dtype == TW_BF16 ? 2 : 4;
  const struct { const void* at; size_t bytes; bool written; } arrays[] = {
      {t.p, n * pb, true},           {t.master, n * 4, true},        {t.g, n * gb, false},
      {t.m, n * sb, true},           {t.v, n * sb, true},            {t.m_scale, blocks * 4, true},
      {t.v_scale, blocks * 4, true}, {t.m_values, n * vb, true},     {t.v_values, n * vb, true}};
  for (const auto& a : arrays) {
    if (!a.at) continue;
    if (!aligned16(a.at)) return TW_ERR_ALIGNMENT;
    const uintptr_t first = reinterpret_cast<uintptr_t>(a.at);
    ranges->push_back({first, first + a.bytes, a.written});
  }
  return TW_OK;
}

tw_status adamw_step(const tw_adamw_tensor* tensors, int32_t count, const tw_adamw_args* args,
                     cudaStream_t stream) {
  if (count < 0 || (count > 0 && !tensors) || !args) return TW_ERR_INVALID_ARG;
  const double scalars[] = {args->lr, args->beta1, args->beta2, args->eps};
  for (double v : scalars)
    if (!std::isfinite(v) || v < 0.0) return TW_ERR_INVALID_ARG;
  if (args->beta1 >= 1.0 || args->beta2 >= 1.0 || (float)args->eps < FLT_MIN)
    return TW_ERR_INVALID_ARG;
  if (!args->step_dev && args->step < 1) return TW_ERR_INVALID_ARG;
  const void* words[] = {args->lr_dev, args->step_dev, args->grad_scale};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return TW_ERR_ALIGNMENT;
  // no exception may leave a C entry
  try {
    std::vector<AdamwRange> ranges;
    ranges.reserve(9 * (size_t)count + 3);
    for (const void* w : words)  // four bytes each, read while the arrays are written
      if (w) ranges.push_back({reinterpret_cast<uintptr_t>(w), reinterpret_cast<uintptr_t>(w) + 4, false});
    for (int32_t i = 0; i < count; ++i) {
      tw_status st = check_adamw_tensor(tensors[i], &ranges);
      if (st != TW_OK) return st;
    }
    std::sort(ranges.begin(), ranges.end(),
              [](const AdamwRange& a, const AdamwRange& b) { return a.first < b.first; });
    // sweep by start: the furthest end of the written and of all ranges so far
    uintptr_t end_written = 0, end_any = 0;
    for (const AdamwRange& r : ranges) {
      if (r.first < (r.written ? end_any : end_written)) return TW_ERR_INVALID_ARG;
      end_any = std::max(end_any, r.last);
      if (r.written) end_written = std::max(end_written, r.last);
    }
  } catch (...) {
    return TW_ERR_UNSUPPORTED;  // no host memory for the list's ranges
  }
  return from_cuda(tw::launch_adamw(tensors, count, *args, stream));
}

// Workspace of the dense training comparator: g, u, h (saved by the forward
// for the backward) then du, dz (backward scratch), each [T][F] bf16.
static size_t dense_train_part(int32_t T, int32_t F) {
  return ((size_t)T * (size_t)F * 2 + 255) & ~size_t(255);
}

size_t dense_ffn_train_workspace_size(int32_t T, int32_t F) {
  if (T < 0 || F <= 0) return 0;
  return 5 * dense_train_part(T, F);
}

size_t dense_ffn_train_saved_bytes(int32_t T, int32_t F) {
  if (T < 0 || F <= 0) return 0;
  return 3 * dense_train_part(T, F);
}

static tw_status check_dense_train(int32_t T, int32_t d, int32_t F, const void* ws,
                                   size_t ws_bytes) {
  if (T < 0 || d <= 0 || F <= 0) return TW_ERR_INVALID_ARG;
  if (d % 32 != 0 || d < 64 || F % kTileW != 0) return TW_ERR_UNSUPPORTED;
  if (T > 0 && !ws) return TW_ERR_INVALID_ARG;
  if (!aligned16(ws)) return TW_ERR_ALIGNMENT;
  if (T > 0 && ws_bytes < 5 * dense_train_part(T, F)) return TW_ERR_WORKSPACE;
  return TW_OK;
}

tw_status dense_ffn_train_forward(const void* x, const void* Wg_t, const void* Wu_t,
                                  const void* Wd, int32_t T, int32_t d, int32_t F, void* ws,
                                  size_t ws_bytes, float* y, int32_t* dev_status,
                                  cudaStream_t stream) {
  tw_status st = check_dense_train(T, d, F, ws, ws_bytes);
  if (st != TW_OK) return st;
  if ((T > 0 && (!x || !y)) || !Wg_t || !Wu_t || !Wd) return TW_ERR_INVALID_ARG;
  const void* ptrs[] = {x, Wg_t, Wu_t, Wd, y};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if (T == 0) return TW_OK;
  uint16_t* base = static_cast<uint16_t*>(ws);
  const size_t part = dense_train_part(T, F) / 2;
  return from_cuda(tw::launch_dense_train_forward(x, Wg_t, Wu_t, Wd, T, d, F, base,
                                                  base + part, base + 2 * part, y, dev_status,
                                                  stream));
}

tw_status dense_ffn_train_backward(const void* x, const void* dy, const void* Wg_t,
                                   const void* Wu_t, const void* Wd, int32_t T, int32_t d,
                                   int32_t F, float l1_lambda, void* ws, size_t ws_bytes,
                                   float* dx, float* dWg_t, float* dWu_t, float* dWd,
                                   int32_t* dev_status, cudaStream_t stream) {
  tw_status st = check_dense_train(T, d, F, ws, ws_bytes);
  if (st != TW_OK) return st;
  if ((T > 0 && (!x || !dy || !dx)) || !Wg_t || !Wu_t || !Wd || !dWg_t || !dWu_t || !dWd)
    return TW_ERR_INVALID_ARG;
  const void* ptrs[] = {x, dy, Wg_t, Wu_t, Wd, dx, dWg_t, dWu_t, dWd};
  for (const void* p : ptrs)
    if (!aligned16(p)) return TW_ERR_ALIGNMENT;
  if (T == 0) {  // no tokens: zero weight gradients
    const size_t b = sizeof(float) * (size_t)F * d;
    cudaError_t e = cudaMemsetAsync(dWg_t, 0, b, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(dWu_t, 0, b, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(dWd, 0, b, stream);
    return from_cuda(e);
  }
  uint16_t* base = static_cast<uint16_t*>(ws);
  const size_t part = dense_train_part(T, F) / 2;
  return from_cuda(tw::launch_dense_train_backward(
      x, dy, Wg_t, Wu_t, Wd, T, d, F, l1_lambda, base, base + part, base + 2 * part,
      base + 3 * part, base + 4 * part, dx, dWg_t, dWu_t, dWd, dev_status, stream));
}

}  // extern "C"
