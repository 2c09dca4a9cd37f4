// Activation checkpoints in 8 bits.
//
// A row is cut into blocks of 32 consecutive columns (SwiGLU rows: of each
// half, gate and up).  A block stores one exponent byte E, the exponent field
// of its largest magnitude as an fp32 number, and per element
//     q = clamp(round_to_nearest_even(x 2^(133 - E)), -127, 127)   (int8)
// which stands for q 2^(E - 133): a microscaled 8-bit integer with a
// power-of-two scale.  The largest magnitude lies in [2^(E-127), 2^(E-126)),
// so its q is at least 64 and every element is off by at most 2^(E - 134)
// (2^(E - 133) where the clamp takes a q of 128).  Scaling by powers of two
// is exact, so the result is the same in any arithmetic of 24 bits or more.
// E = 255 (a NaN or an infinity in the block): every element reads back as
// NaN, so that nothing non-finite is lost.
//
// Everything here is bound by the bytes it moves: each element is read once
// and written once per form (bf16 or fp32 in, 8 bits + 1/32 byte out).
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kBlk = MOE_CKPT_BLOCK;

__device__ __forceinline__ int live_rows(const int32_t* n_rows, int rows) {
  return n_rows != nullptr ? max(0, min(rows, *n_rows)) : rows;
}

// 2^(127 - E): takes the block's largest magnitude into [1, 2).  E = 255: 0.
__device__ __forceinline__ float ckpt_inv_scale(uint32_t e) {
  return __uint_as_float(e < 254u ? (254u - e) << 23 : (e == 254u ? 0x00400000u : 0u));
}
// 2^(E - 133), subnormal for E <= 6; E = 255: NaN.
__device__ __forceinline__ float ckpt_scale(uint32_t e) {
  return __uint_as_float(e >= 255u ? 0x7fc00000u : (e >= 7u ? (e - 6u) << 23 : 1u << (16u + e)));
}
__device__ __forceinline__ int ckpt_q(float v, float inv) {
  return max(-127, min(127, __float2int_rn(v * inv * 64.0f)));
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// sigmoid(x) and sigmoid(-x), neither by a difference: with z = exp(-|x|)
// they are 1 / (1 + z) and z / (1 + z).  The divisor is in [1, 2], where the
// approximate division is within 2 ulp.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& ns) {
  const float z = __expf(-fabsf(x));
  const float p = __fdividef(1.0f, 1.0f + z);
  const float m = z * p;
  s = x < 0.0f ? m : p;
  ns = x < 0.0f ? p : m;
}

// GELU (tanh form) as v sigmoid(w(v)) with w = 2 sqrt(2/pi) (v + 0.044715 v^3):
// 0.5 (1 + tanh(w / 2)) = sigmoid(w), without the cancellation at negative v.
// Its derivative is sigmoid(w) + v sigmoid(w) sigmoid(-w) w'(v).
constexpr float kGeluW = 1.5957691216057308f;  // 2 sqrt(2/pi)
__device__ __forceinline__ float gelu_sig(float v) {
  float s, ns;
  sigmoid_pair(kGeluW * fmaf(0.044715f * v, v * v, v), s, ns);
  return v * s;
}
__device__ __forceinline__ void gelu_sig_grad(float v, float& a, float& da) {
  // beyond |v| = 20 sigmoid(-|w|) is 0 in fp32; the clamp keeps w' finite there (NaN passes through)
  const float c = fabsf(v) > 20.0f ? copysignf(20.0f, v) : v;
  float s, ns;
  sigmoid_pair(kGeluW * fmaf(0.044715f * c, c * c, c), s, ns);
  a = v * s;
  da = fmaf(c * s * ns, kGeluW * fmaf(3.0f * 0.044715f * c, c, 1.0f), s);
}
__device__ __forceinline__ float swiglu(float g, float u) {
  float s, ns;
  sigmoid_pair(g, s, ns);
  return g * s * u;
}
__device__ __forceinline__ void swiglu_grad(float g, float u, float& a, float& dg, float& du) {
  float s, ns;
  sigmoid_pair(g, s, ns);
  du = g * s;                        // da / du = SiLU(g)
  a = du * u;
  dg = u * s * fmaf(g, ns, 1.0f);    // da / dg = u SiLU'(g)
}

// ------------------------------------------------ any width: warp per block
template <typename T>
__global__ void __launch_bounds__(256) ckpt_quantize_kernel(const T* __restrict__ src, const int32_t* n_rows, int rows,
                                                            int cols, int nb, int8_t* __restrict__ q,
                                                            uint8_t* __restrict__ e) {
  const int lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(live_rows(n_rows, rows)) * nb;
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long i = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < units;
       i += step) {
    const long long r = i / nb;
    const int c = static_cast<int>(i - r * nb) * kBlk + lane;
    const float v = c < cols ? to_f32(src[r * cols + c]) : 0.0f;
    const uint32_t ex = __reduce_max_sync(0xffffffffu, abs_bits(v)) >> 23;
    if (c < cols) q[r * cols + c] = static_cast<int8_t>(ckpt_q(v, ckpt_inv_scale(ex)));
    if (lane == 0) e[i] = static_cast<uint8_t>(ex);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_dequantize_kernel(const int8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ e,
                                                              const int32_t* __restrict__ row_index,
                                                              const int32_t* n_rows, int rows, int src_rows, int cols,
                                                              int nb, T* __restrict__ dst, int* status) {
  const int lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(live_rows(n_rows, rows)) * nb;
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long i = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < units;
       i += step) {
    const long long r = i / nb;
    const int b = static_cast<int>(i - r * nb);
    const int c = b * kBlk + lane;
    const long long sr = row_index != nullptr ? row_index[r] : r;
    const bool ok = sr >= 0 && sr < src_rows;
    if (!ok && lane == 0) set_status(status, MOE_DEVERR_BAD_ROW_TOKEN);
    if (c < cols)
      dst[r * cols + c] =
          from_f32<T>(ok ? static_cast<float>(q[sr * cols + c]) * ckpt_scale(e[sr * nb + b]) : 0.0f);
  }
}

template <typename TS, typename TD, bool SWIGLU>
__global__ void __launch_bounds__(256) act_save_kernel(const TS* __restrict__ h, const int32_t* n_rows, int rows,
                                                       int I, int nb, TD* __restrict__ a, int8_t* __restrict__ q,
                                                       uint8_t* __restrict__ e) {
  constexpr int H = SWIGLU ? 2 : 1;
  const int lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(live_rows(n_rows, rows)) * nb;
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long i = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < units;
       i += step) {
    const long long r = i / nb;
    const int b = static_cast<int>(i - r * nb);
    const int c = b * kBlk + lane;
    float v[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
      v[j] = c < I ? to_f32(h[(r * H + j) * I + c]) : 0.0f;
      const uint32_t ex = __reduce_max_sync(0xffffffffu, abs_bits(v[j])) >> 23;
      if (c < I) q[(r * H + j) * I + c] = static_cast<int8_t>(ckpt_q(v[j], ckpt_inv_scale(ex)));
      if (lane == 0) e[(r * H + j) * nb + b] = static_cast<uint8_t>(ex);
    }
    if (c < I) {
      if constexpr (SWIGLU) a[r * I + c] = from_f32<TD>(swiglu(v[0], v[1]));
      else a[r * I + c] = from_f32<TD>(gelu_sig(v[0]));
    }
  }
}

// Block per row, so that the row's dot product <da, a> stays inside a block.
template <typename TS, typename TD, bool SWIGLU>
__global__ void __launch_bounds__(256) act_backward_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e,
                                                           const TS* __restrict__ da, const float* __restrict__ row_w,
                                                           const int32_t* n_rows, int rows, int I, int nb,
                                                           TD* __restrict__ dh, TD* __restrict__ wa,
                                                           float* __restrict__ dw) {
  constexpr int H = SWIGLU ? 2 : 1;
  __shared__ float s_part[8];
  const int n = live_rows(n_rows, rows);
  for (long long r = blockIdx.x; r < n; r += gridDim.x) {
    const float w = row_w != nullptr ? row_w[r] : 1.0f;
    float dot = 0.0f;
    for (int c = threadIdx.x; c < I; c += blockDim.x) {
      const float g = to_f32(da[r * I + c]);
      float v[H], a, d[H];
#pragma unroll
      for (int j = 0; j < H; ++j)
        v[j] = static_cast<float>(q[(r * H + j) * I + c]) * ckpt_scale(e[(r * H + j) * nb + c / kBlk]);
      if constexpr (SWIGLU) swiglu_grad(v[0], v[1], a, d[0], d[1]);
      else gelu_sig_grad(v[0], a, d[0]);
#pragma unroll
      for (int j = 0; j < H; ++j) dh[(r * H + j) * I + c] = from_f32<TD>(w * g * d[j]);
      if (wa != nullptr) wa[r * I + c] = from_f32<TD>(w * a);
      dot = fmaf(g, a, dot);
    }
    if (dw != nullptr) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        float t = 0.0f;
        for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) t += s_part[i];
        dw[r] = t;
      }
      __syncthreads();
    }
  }
}

inline int warp_grid(long long units) {
  return static_cast<int>(std::max<long long>(1, std::min<long long>((units + 7) / 8, 8ll * num_sms())));
}
inline int blocks_of(int cols) { return (cols + kBlk - 1) / kBlk; }

}  // namespace

cudaError_t launch_ckpt_quantize(int dtype, const void* src, const int32_t* n_rows, int rows, int cols, int8_t* q,
                                 uint8_t* e, cudaStream_t s) {
  const int nb = blocks_of(cols), grid = warp_grid(static_cast<long long>(rows) * nb);
  if (dtype == MOE_DTYPE_BF16)
    ckpt_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(src), n_rows, rows, cols, nb, q, e);
  else
    ckpt_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(src), n_rows, rows, cols, nb, q, e);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_dequantize(int dtype, const int8_t* q, const uint8_t* e, const int32_t* row_index,
                                   const int32_t* n_rows, int rows, int src_rows, int cols, void* dst, int* status,
                                   cudaStream_t s) {
  const int nb = blocks_of(cols), grid = warp_grid(static_cast<long long>(rows) * nb);
  if (dtype == MOE_DTYPE_BF16)
    ckpt_dequantize_kernel<<<grid, 256, 0, s>>>(q, e, row_index, n_rows, rows, src_rows, cols, nb,
                                                static_cast<__nv_bfloat16*>(dst), status);
  else
    ckpt_dequantize_kernel<<<grid, 256, 0, s>>>(q, e, row_index, n_rows, rows, src_rows, cols, nb,
                                                static_cast<float*>(dst), status);
  return cudaGetLastError();
}

namespace {

template <typename TS, typename TD>
void run_save(bool sw, const void* h, const int32_t* n_rows, int rows, int I, void* a, int8_t* q, uint8_t* e,
              cudaStream_t s) {
  const int nb = blocks_of(I), grid = warp_grid(static_cast<long long>(rows) * nb);
  if (sw)
    act_save_kernel<TS, TD, true><<<grid, 256, 0, s>>>(static_cast<const TS*>(h), n_rows, rows, I, nb,
                                                       static_cast<TD*>(a), q, e);
  else
    act_save_kernel<TS, TD, false><<<grid, 256, 0, s>>>(static_cast<const TS*>(h), n_rows, rows, I, nb,
                                                        static_cast<TD*>(a), q, e);
}

template <typename TS, typename TD>
void run_backward(bool sw, const int8_t* q, const uint8_t* e, const void* da, const float* row_w,
                  const int32_t* n_rows, int rows, int I, void* dh, void* wa, float* dw, cudaStream_t s) {
  const int nb = blocks_of(I), grid = std::min(rows, 8 * num_sms());
  if (sw)
    act_backward_kernel<TS, TD, true><<<grid, 256, 0, s>>>(q, e, static_cast<const TS*>(da), row_w, n_rows, rows, I,
                                                           nb, static_cast<TD*>(dh), static_cast<TD*>(wa), dw);
  else
    act_backward_kernel<TS, TD, false><<<grid, 256, 0, s>>>(q, e, static_cast<const TS*>(da), row_w, n_rows, rows, I,
                                                            nb, static_cast<TD*>(dh), static_cast<TD*>(wa), dw);
}

}  // namespace

cudaError_t launch_act_save(int dtype, int src_dtype, bool sw, const void* h, const int32_t* n_rows, int rows, int I,
                            void* a, int8_t* q, uint8_t* e, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (src_dtype == MOE_DTYPE_BF16) {
    if (dtype == MOE_DTYPE_BF16) run_save<bf, bf>(sw, h, n_rows, rows, I, a, q, e, s);
    else run_save<bf, float>(sw, h, n_rows, rows, I, a, q, e, s);
  } else {
    if (dtype == MOE_DTYPE_BF16) run_save<float, bf>(sw, h, n_rows, rows, I, a, q, e, s);
    else run_save<float, float>(sw, h, n_rows, rows, I, a, q, e, s);
  }
  return cudaGetLastError();
}

cudaError_t launch_act_backward(int dtype, int src_dtype, bool sw, const int8_t* q, const uint8_t* e, const void* da,
                                const float* row_w, const int32_t* n_rows, int rows, int I, void* dh, void* wa,
                                float* dw, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (src_dtype == MOE_DTYPE_BF16) {
    if (dtype == MOE_DTYPE_BF16) run_backward<bf, bf>(sw, q, e, da, row_w, n_rows, rows, I, dh, wa, dw, s);
    else run_backward<bf, float>(sw, q, e, da, row_w, n_rows, rows, I, dh, wa, dw, s);
  } else {
    if (dtype == MOE_DTYPE_BF16) run_backward<float, bf>(sw, q, e, da, row_w, n_rows, rows, I, dh, wa, dw, s);
    else run_backward<float, float>(sw, q, e, da, row_w, n_rows, rows, I, dh, wa, dw, s);
  }
  return cudaGetLastError();
}

}  // namespace moe
