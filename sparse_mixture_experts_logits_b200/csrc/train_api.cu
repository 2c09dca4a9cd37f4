// C ABI of the experts' step-by-step operators: the matrix products grouped
// by expert and the 8-bit activation checkpoints (see moe_b200.h).
#include "api_util.cuh"

using namespace moe;

namespace {

moe_status_t check_grouped(int G, int N, int K, int rows, int dtype) {
  if (G < 1 || N < 1 || K < 1 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(dtype) || G > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(N) * K >= (1ll << 40) / G) return MOE_ERR_UNSUPPORTED;
  if (rows >= (1 << 30) || N >= (1 << 24) || K >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  // The forward counts the weight rows of all experts in 32 bits, up to a tile behind the last one (its boxes'
  // coordinates): past 2^31 they are no positions in the tensor, and loads at them faulted.
  if (static_cast<long long>(G) * N >= (1ll << 31) - 1024) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t check_out(int dtype, int out_dtype) {
  if (!is_dtype(out_dtype)) return MOE_ERR_UNSUPPORTED;
  return dtype == MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_F32 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Bytes of a call's workspace: the head (status word, tile counters) and what
// the tensor-core path of the product needs.
size_t grouped_ws(int dir, int G, int N, int K, int dtype) {
  return grouped_tc_ok(dtype, N, K) ? grouped_tc_workspace(dir, G, N, K) : kAlign;
}

// moe_grouped_wgrad: that, and (tensor cores) the bias gradient's partial sums behind it.
struct WgradWs { size_t part, total; };
WgradWs wgrad_layout(int G, int N, int K, int rows, int dtype) {
  Carve c;
  WgradWs L;
  c.take(grouped_ws(kGroupedWgrad, G, N, K, dtype));
  const int shares = grouped_tc_ok(dtype, N, K) ? grouped_colsum_shares(G, rows, N) : 1;
  L.part = c.take(shares > 1 ? static_cast<size_t>(shares) * G * N * 4 : 0);
  L.total = c.off;
  return L;
}

// Clears the status word first (in the launches themselves).
moe_status_t run_grouped(const GroupedLaunch& L, void* ws, cudaStream_t s) {
  if (grouped_tc_ok(L.dtype, L.N, L.K)) return cuda_status(launch_grouped_tc(L, ws, s));
  return cuda_status(launch_grouped_simt(L, static_cast<int*>(ws), s));
}

// The arguments that the two row products share.
moe_status_t check_rows_call(const void* a, const void* w, const int32_t* offsets, int G, int N, int K, int rows,
                             int dtype, int out_dtype, const void* out, const void* ws, size_t ws_bytes) {
  MOE_TRY(check_grouped(G, N, K, rows, dtype));
  MOE_TRY(check_out(dtype, out_dtype));
  if (rows == 0) return MOE_OK;
  if (!a || !w || !offsets || !out || !ws || !aligned_ws(ws)) return MOE_ERR_INVALID_ARG;
  if (grouped_tc_ok(dtype, N, K) && (!al16(a) || !al16(w) || !al16(out))) return MOE_ERR_INVALID_ARG;
  return ws_bytes < grouped_ws(kGroupedFwd, G, N, K, dtype) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

moe_status_t check_act(int rows, int I, int act, int dtype, int src_dtype) {
  if (rows < 0 || I < 1) return MOE_ERR_INVALID_ARG;
  if (act != MOE_ACT_GELU_TANH && act != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(dtype) || !is_dtype(src_dtype)) return MOE_ERR_UNSUPPORTED;
  return rows >= (1 << 30) || I >= (1 << 30) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_grouped_workspace_size(int G, int N, int K, int rows, int dtype) {
  return check_grouped(G, N, K, rows, dtype) == MOE_OK ? grouped_ws(kGroupedFwd, G, N, K, dtype) : 0;
}

moe_status_t moe_grouped_gemm(const void* x, const void* w, const void* bias, const int32_t* offsets, int G, int N,
                              int K, int rows, int dtype, int out_dtype, void* y, void* ws, size_t ws_bytes,
                              void* stream) {
  MOE_TRY(check_rows_call(x, w, offsets, G, N, K, rows, dtype, out_dtype, y, ws, ws_bytes));
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_device());
  GroupedLaunch L{};
  L.dir = kGroupedFwd;
  L.dtype = dtype; L.out_dtype = out_dtype;
  L.G = G; L.N = N; L.K = K; L.rows = rows;
  L.offsets = offsets;
  L.x = x; L.w = w; L.bias = bias; L.out = y;
  return run_grouped(L, ws, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_grouped_dgrad(const void* dy, const void* w, const int32_t* offsets, int G, int N, int K, int rows,
                               int dtype, int out_dtype, void* dx, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_rows_call(dy, w, offsets, G, N, K, rows, dtype, out_dtype, dx, ws, ws_bytes));
  if (rows == 0) return MOE_OK;
  MOE_TRY(check_device());
  GroupedLaunch L{};
  L.dir = kGroupedDgrad;
  L.dtype = dtype; L.out_dtype = out_dtype;
  L.G = G; L.N = N; L.K = K; L.rows = rows;
  L.offsets = offsets;
  L.dy = dy; L.w = w; L.out = dx;
  return run_grouped(L, ws, static_cast<cudaStream_t>(stream));
}

size_t moe_grouped_wgrad_workspace_size(int G, int N, int K, int rows, int dtype) {
  return check_grouped(G, N, K, rows, dtype) == MOE_OK ? wgrad_layout(G, N, K, rows, dtype).total : 0;
}

moe_status_t moe_grouped_wgrad(const void* x, const void* dy, const int32_t* offsets, int G, int N, int K, int rows,
                               int dtype, int accumulate, float* dw, float* db, void* ws, size_t ws_bytes,
                               void* stream) {
  MOE_TRY(check_grouped(G, N, K, rows, dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!dw) return MOE_ERR_INVALID_ARG;
  if (rows == 0) {
    if (accumulate) return MOE_OK;
    MOE_TRY(check_device());
    MOE_CUDA(cudaMemsetAsync(dw, 0, static_cast<size_t>(G) * N * K * 4, s));
    if (db) MOE_CUDA(cudaMemsetAsync(db, 0, static_cast<size_t>(G) * N * 4, s));
    return MOE_OK;
  }
  if (!x || !dy || !offsets || !ws || !aligned_ws(ws)) return MOE_ERR_INVALID_ARG;
  if (grouped_tc_ok(dtype, N, K) && (!al16(x) || !al16(dy) || !al16(dw))) return MOE_ERR_INVALID_ARG;
  const WgradWs W = wgrad_layout(G, N, K, rows, dtype);
  if (ws_bytes < W.total) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_device());
  GroupedLaunch L{};
  L.dir = kGroupedWgrad;
  L.dtype = dtype; L.out_dtype = MOE_DTYPE_F32;
  L.G = G; L.N = N; L.K = K; L.rows = rows;
  L.offsets = offsets;
  L.x = x; L.dy = dy; L.out = dw;
  L.accumulate = accumulate != 0;
  L.db = db;
  L.part = at<float*>(ws, W.part);
  return run_grouped(L, ws, s);
}

int moe_ckpt_blocks(int cols) { return cols < 1 ? 0 : (cols - 1) / MOE_CKPT_BLOCK + 1; }

moe_status_t moe_ckpt_quantize(const void* src, const int32_t* n_rows, int rows, int cols, int dtype, int8_t* q,
                               uint8_t* e, void* stream) {
  MOE_TRY(check_act(rows, cols, MOE_ACT_GELU_TANH, dtype, dtype));
  if (rows == 0) return MOE_OK;
  if (!src || !q || !e) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_device());
  return cuda_status(launch_ckpt_quantize(dtype, src, n_rows, rows, cols, q, e, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_ckpt_dequantize(const int8_t* q, const uint8_t* e, const int32_t* row_index, const int32_t* n_rows,
                                 int rows, int src_rows, int cols, int dtype, void* dst, int32_t* device_status,
                                 void* stream) {
  MOE_TRY(check_act(rows, cols, MOE_ACT_GELU_TANH, dtype, dtype));
  if (src_rows < 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if ((src_rows > 0 && (!q || !e)) || !dst) return MOE_ERR_INVALID_ARG;
  if (row_index == nullptr && rows > src_rows) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_device());
  return cuda_status(launch_ckpt_dequantize(dtype, q, e, row_index, n_rows, rows, src_rows, cols, dst, device_status,
                                            static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_act_save(const void* h, const int32_t* n_rows, int rows, int I, int act, int dtype, int src_dtype,
                          void* a, int8_t* q, uint8_t* e, void* stream) {
  MOE_TRY(check_act(rows, I, act, dtype, src_dtype));
  if (rows == 0) return MOE_OK;
  if (!h || !a || !q || !e) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_device());
  return cuda_status(launch_act_save(dtype, src_dtype, act == MOE_ACT_SWIGLU, h, n_rows, rows, I, a, q, e,
                                     static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_act_backward(const int8_t* q, const uint8_t* e, const void* da, const float* row_w,
                              const int32_t* n_rows, int rows, int I, int act, int dtype, int src_dtype, void* dh,
                              void* wa, float* dw, void* stream) {
  MOE_TRY(check_act(rows, I, act, dtype, src_dtype));
  if (rows == 0) return MOE_OK;
  if (!q || !e || !da || !dh) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_device());
  return cuda_status(launch_act_backward(dtype, src_dtype, act == MOE_ACT_SWIGLU, q, e, da, row_w, n_rows, rows, I,
                                         dh, wa, dw, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
