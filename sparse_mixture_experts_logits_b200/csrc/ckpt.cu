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
// Measured on a B200 whose copies reach 6.5 TB/s, bf16: SwiGLU of 32768 x
// 2048 saved in 91 us (6.0 TB/s), its backward 109 us (6.2); GELU of 16384 x
// 8192 113 and 160 us (5.9 TB/s); rows of 8192 x 5120 kept in 27 us and read
// back four times in 69 us (writes; a plain fill of those bytes takes 88).
// Widths that are no multiple of 8 run at about half these rates.
#include <algorithm>

#include "ckpt.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

__device__ __forceinline__ int live_rows(const int32_t* n_rows, int rows) {
  return n_rows != nullptr ? max(0, min(rows, *n_rows)) : rows;
}

// s = sigmoid(x) and d = s (1 - s) from y = x log2(e), without a difference:
// with z = exp(-x) they are s = 1 / (1 + z) and (z s) s.  The hardware's
// exponential (2 ulp) and reciprocal (1 ulp, 0 instead of a subnormal); the
// clamp at y = -127 keeps z finite where s is 0.  (A NaN is clamped too: it
// reaches the results through the factors x.)
__device__ __forceinline__ void sigmoid_of(F2 y, F2& s, F2& d) {
  float y0, y1, z0, z1, p0, p1;
  un2(y, y0, y1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z0) : "f"(-fmaxf(y0, -127.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z1) : "f"(-fmaxf(y1, -127.0f)));
  const F2 z = f2(z0, z1);
  un2(z + f2(1.0f), p0, p1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p0) : "f"(p0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p1) : "f"(p1));
  s = f2(p0, p1);
  d = z * s * s;
}
constexpr float kLog2e = 1.4426950408889634f;

// GELU (tanh form) as v sigmoid(w(v)) with w = 2 sqrt(2/pi) (v + 0.044715 v^3):
// 0.5 (1 + tanh(w / 2)) = sigmoid(w), without the cancellation at negative v.
// Its derivative is sigmoid(w) + v sigmoid(w) sigmoid(-w) w'(v).  The cubic's
// coefficients carry the log2(e) of sigmoid_of.
constexpr float kGeluW = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluC = 0.044715f;
__device__ __forceinline__ F2 gelu_sig(F2 v) {
  F2 s, d;
  sigmoid_of(v * fma2(f2(kGeluW * kGeluC * kLog2e), v * v, f2(kGeluW * kLog2e)), s, d);
  return v * s;
}
__device__ __forceinline__ void gelu_sig_grad(F2 v, F2& a, F2& da) {
  F2 s, d;
  const F2 q = v * v;
  sigmoid_of(v * fma2(f2(kGeluW * kGeluC * kLog2e), q, f2(kGeluW * kLog2e)), s, d);
  a = v * s;
  // w' is kept finite where v^2 overflows: d is next to 0 there
  float w0, w1;
  un2(fma2(f2(3.0f * kGeluW * kGeluC), q, f2(kGeluW)), w0, w1);
  da = fma2(v * d, f2(fminf(w0, 1e18f), fminf(w1, 1e18f)), s);
}
__device__ __forceinline__ F2 swiglu(F2 g, F2 u) {
  F2 s, d;
  sigmoid_of(g * f2(kLog2e), s, d);
  return g * s * u;
}
__device__ __forceinline__ void swiglu_grad(F2 g, F2 u, F2& a, F2& dg, F2& du) {
  F2 s, d;
  sigmoid_of(g * f2(kLog2e), s, d);
  du = g * s;                // da / du = SiLU(g)
  a = du * u;
  dg = u * fma2(g, d, s);    // da / dg = u SiLU'(g)
}

// ------------------------------------------- any width and alignment
// A warp takes kB blocks of 32 columns of a row at a time, a lane one column
// of each: every access is a value wide, so that nothing is asked of the
// width or the alignment, and kB (times the halves) loads are in flight.
// FULL: all of the kB blocks lie inside the row, and nothing is compared.
constexpr int kB = 8;

// This lane's kB values, from its first column on (`left`: columns from there
// to the row's end; 0 behind it).
template <bool FULL, typename T>
__device__ __forceinline__ void load_blocks(const T* __restrict__ p, int left, float (&v)[kB]) {
#pragma unroll
  for (int j = 0; j < kB; ++j) v[j] = FULL || 32 * j < left ? to_f32(p[32 * j]) : 0.0f;
}
template <bool FULL, typename T>
__device__ __forceinline__ void store_blocks(T* __restrict__ p, int left, const float (&v)[kB]) {
#pragma unroll
  for (int j = 0; j < kB; ++j)
    if (FULL || 32 * j < left) p[32 * j] = from_f32<T>(v[j]);
}
// Keeps them: q from this lane's first column on and, lane j, the exponent of
// block j.  Rounded as in keep8, with the same long way for the rare rest.
template <bool FULL>
__device__ __forceinline__ void keep_blocks(const float (&v)[kB], int left, int blocks, int lane,
                                            int8_t* __restrict__ q, uint8_t* __restrict__ e) {
  uint32_t mine = 0, ex[kB], b[kB];
  bool odd = false;
#pragma unroll
  for (int j = 0; j < kB; ++j) {
    ex[j] = __reduce_max_sync(0xffffffffu, abs_bits(v[j])) >> 23;
    if (lane == j) mine = ex[j];
    b[j] = __float_as_uint(fmaf(v[j], __uint_as_float((260u - ex[j]) << 23), 12582912.0f));
    odd |= (b[j] & 0xffu) == 0x80u || ex[j] - 6u > 248u;
  }
  if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const float t = fminf(fmaxf(v[j] * ckpt_inv_scale(ex[j]), -127.0f / 64.0f), 127.0f / 64.0f);
      b[j] = ex[j] == 255u ? 0u : __float_as_uint(fmaf(t, 64.0f, 12582912.0f));
    }
  }
#pragma unroll
  for (int j = 0; j < kB; ++j)
    if (FULL || 32 * j < left) q[32 * j] = static_cast<int8_t>(b[j]);
  if (lane < blocks) e[lane] = static_cast<uint8_t>(mine);
}
// The kept values of those columns (0 where `ok` is false).
template <bool FULL>
__device__ __forceinline__ void read_blocks(const int8_t* __restrict__ q, const uint8_t* __restrict__ e, bool ok,
                                            int left, int blocks, int lane, float (&v)[kB]) {
  int k[kB];
#pragma unroll
  for (int j = 0; j < kB; ++j) k[j] = ok && (FULL || 32 * j < left) ? q[32 * j] : 0;
  const float s = ckpt_scale(ok && lane < blocks ? e[lane] : 0u);
#pragma unroll
  for (int j = 0; j < kB; ++j)
    v[j] = (__uint_as_float(0x4B000080u + static_cast<uint32_t>(k[j])) - 8388736.0f) * __shfl_sync(0xffffffffu, s, j);
}

// This warp's pieces of a batch: `chunks` of kB blocks a row, every
// gridDim x 8-th piece, stepped without a division.
struct Walk {
  long long r;
  int ch, dq, dr, chunks;
  __device__ explicit Walk(int nb) : chunks((nb + kB - 1) / kB) {
    const int start = blockIdx.x * 8 + (threadIdx.x >> 5), step = gridDim.x * 8;
    r = start / chunks;
    ch = start % chunks;
    dq = step / chunks;
    dr = step % chunks;
  }
  __device__ void next() {
    r += dq;
    ch += dr;
    if (ch >= chunks) { ch -= chunks; ++r; }
  }
};
// Calls f(true) for a piece inside the row and f(false) for the row's end
// (as types: the branch is the warp's).
template <bool V> struct Bool { static constexpr bool value = V; };
template <typename F>
__device__ __forceinline__ void full_or_not(bool full, F&& f) {
  if (full) f(Bool<true>()); else f(Bool<false>());
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_quantize_kernel(const T* __restrict__ src, const int32_t* n_rows, int rows,
                                                            int cols, int nb, int8_t* __restrict__ q,
                                                            uint8_t* __restrict__ e) {
  const int lane = threadIdx.x & 31, n = live_rows(n_rows, rows);
  for (Walk w(nb); w.r < n; w.next()) {
    const int b0 = w.ch * kB, c0 = b0 * kBlk + lane;
    full_or_not((b0 + kB) * kBlk <= cols, [&](auto full) {
      constexpr bool F = decltype(full)::value;
      float v[kB];
      load_blocks<F>(src + w.r * cols + c0, cols - c0, v);
      keep_blocks<F>(v, cols - c0, nb - b0 < kB ? nb - b0 : kB, lane, q + w.r * cols + c0, e + w.r * nb + b0);
    });
  }
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_dequantize_kernel(const int8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ e,
                                                              const int32_t* __restrict__ row_index,
                                                              const int32_t* n_rows, int rows, int src_rows, int cols,
                                                              int nb, T* __restrict__ dst, int* status) {
  const int lane = threadIdx.x & 31, n = live_rows(n_rows, rows);
  for (Walk w(nb); w.r < n; w.next()) {
    const int b0 = w.ch * kB, c0 = b0 * kBlk + lane;
    const long long sr = row_index != nullptr ? row_index[w.r] : w.r;
    const bool ok = sr >= 0 && sr < src_rows;
    if (!ok && lane == 0) set_status(status, MOE_DEVERR_BAD_ROW_TOKEN);
    full_or_not((b0 + kB) * kBlk <= cols, [&](auto full) {
      constexpr bool F = decltype(full)::value;
      float v[kB];
      read_blocks<F>(q + (ok ? sr : 0) * cols + c0, e + (ok ? sr : 0) * nb + b0, ok, cols - c0,
                     nb - b0 < kB ? nb - b0 : kB, lane, v);
      store_blocks<F>(dst + w.r * cols + c0, cols - c0, v);
    });
  }
}

template <typename TS, typename TD, bool SWIGLU>
__global__ void __launch_bounds__(256) act_save_kernel(const TS* __restrict__ h, const int32_t* n_rows, int rows,
                                                       int I, int nb, TD* __restrict__ a, int8_t* __restrict__ q,
                                                       uint8_t* __restrict__ e) {
  constexpr int H = SWIGLU ? 2 : 1;
  const int lane = threadIdx.x & 31, n = live_rows(n_rows, rows);
  for (Walk w(nb); w.r < n; w.next()) {
    const int b0 = w.ch * kB, c0 = b0 * kBlk + lane;
    full_or_not((b0 + kB) * kBlk <= I, [&](auto full) {
      constexpr bool F = decltype(full)::value;
      const int left = I - c0, blocks = nb - b0 < kB ? nb - b0 : kB;
      float v[H][kB], o[kB];
#pragma unroll
      for (int m = 0; m < H; ++m) load_blocks<F>(h + (w.r * H + m) * I + c0, left, v[m]);
#pragma unroll
      for (int m = 0; m < H; ++m)
        keep_blocks<F>(v[m], left, blocks, lane, q + (w.r * H + m) * I + c0, e + (w.r * H + m) * nb + b0);
#pragma unroll
      for (int j = 0; j < kB; j += 2) {
        const F2 h0 = f2(v[0][j], v[0][j + 1]);
        if constexpr (SWIGLU) un2(swiglu(h0, f2(v[H - 1][j], v[H - 1][j + 1])), o[j], o[j + 1]);
        else un2(gelu_sig(h0), o[j], o[j + 1]);
      }
      store_blocks<F>(a + w.r * I + c0, left, o);
    });
  }
}

// A row's pieces are spread over `wpr` warps of a block (1, or all 8 where
// rows are few), so that its dot product <da, a> needs one block at most.
template <typename TS, typename TD, bool SWIGLU>
__global__ void __launch_bounds__(256) act_backward_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e,
                                                           const TS* __restrict__ da, const float* __restrict__ row_w,
                                                           const int32_t* n_rows, int rows, int I, int nb, int wpr,
                                                           TD* __restrict__ dh, TD* __restrict__ wa,
                                                           float* __restrict__ dw) {
  constexpr int H = SWIGLU ? 2 : 1;
  __shared__ float s_part[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunks = (nb + kB - 1) / kB;
  const int n = live_rows(n_rows, rows), per = 8 / wpr, part = warp % wpr;
  for (long long r0 = static_cast<long long>(blockIdx.x) * per; r0 < n; r0 += static_cast<long long>(gridDim.x) * per) {
    const long long r = r0 + warp / wpr;
    const bool live = r < n;
    const F2 w = f2(live && row_w != nullptr ? row_w[r] : 1.0f);
    F2 dot2 = f2(0.0f);
    for (int ch = part; live && ch < chunks; ch += wpr) {
      const int b0 = ch * kB, c0 = b0 * kBlk + lane;
      full_or_not((b0 + kB) * kBlk <= I, [&](auto full) {
        constexpr bool F = decltype(full)::value;
        const int left = I - c0, blocks = nb - b0 < kB ? nb - b0 : kB;
        float g[kB], v[H][kB], o[kB];
        load_blocks<F>(da + r * I + c0, left, g);
#pragma unroll
        for (int m = 0; m < H; ++m)
          read_blocks<F>(q + (r * H + m) * I + c0, e + (r * H + m) * nb + b0, true, left, blocks, lane, v[m]);
#pragma unroll
        for (int j = 0; j < kB; j += 2) {
          const F2 h0 = f2(v[0][j], v[0][j + 1]), gj = f2(g[j], g[j + 1]);
          F2 a, d[2];
          if constexpr (SWIGLU) swiglu_grad(h0, f2(v[H - 1][j], v[H - 1][j + 1]), a, d[0], d[1]);
          else gelu_sig_grad(h0, a, d[0]);
          dot2 = fma2(gj, a, dot2);
          const F2 wg = w * gj;
          un2(w * a, o[j], o[j + 1]);
#pragma unroll
          for (int m = 0; m < H; ++m) un2(d[m] * wg, v[m][j], v[m][j + 1]);
        }
#pragma unroll
        for (int m = 0; m < H; ++m) store_blocks<F>(dh + (r * H + m) * I + c0, left, v[m]);
        if (wa != nullptr) store_blocks<F>(wa + r * I + c0, left, o);
      });
    }
    if (dw != nullptr) {
      float dot, dot1;
      un2(dot2, dot, dot1);
      dot += dot1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (wpr > 1) {
        if (lane == 0) s_part[warp] = dot;
        __syncthreads();
        dot = 0.0f;
        for (int i = 0; i < wpr; ++i) dot += s_part[warp - part + i];
        __syncthreads();
      }
      if (live && part == 0 && lane == 0) dw[r] = dot;
    }
  }
}

// ------------------------- widths that are a multiple of 8: 16-byte accesses
// A thread takes 8 consecutive columns, four neighbouring threads a block of
// 32; `tx` = 2^lx threads (4 to 256) run along a row and the 256 / tx rows of a
// thread block step through the batch together.  kU column steps are loaded
// before any is used, which keeps 48 to 128 bytes a thread in flight.  Results
// go out with the streaming hint: nothing reads them again from the caches
// before the next kernel.
template <typename T> struct Vec8;  // 8 values as they lie in memory
template <> struct Vec8<__nv_bfloat16> { uint4 a; };
template <> struct Vec8<float> { float4 a, b; };
__device__ __forceinline__ Vec8<__nv_bfloat16> load8(const __nv_bfloat16* p) {
  return {*reinterpret_cast<const uint4*>(p)};
}
__device__ __forceinline__ Vec8<float> load8(const float* p) {
  const float4* q = reinterpret_cast<const float4*>(p);
  return {q[0], q[1]};
}
__device__ __forceinline__ void unpack8(const Vec8<__nv_bfloat16>& v, float* f) { bf16x8_to_f32(v.a, f); }
__device__ __forceinline__ void unpack8(const Vec8<float>& v, float* f) {
  f[0] = v.a.x; f[1] = v.a.y; f[2] = v.a.z; f[3] = v.a.w;
  f[4] = v.b.x; f[5] = v.b.y; f[6] = v.b.z; f[7] = v.b.w;
}
// Columns c .. c + 7 of a row of `cols` (every lane of the warp takes part;
// `on`: the row exists).  fp32: 32 bytes a lane in two stores, whose halves
// neighbouring lanes exchange so that each store fills whole 32-byte sectors.
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int cols, bool on, const float* f) {
  if (on && c < cols) __stcs(reinterpret_cast<uint4*>(row + c), f32_to_bf16x8(f));
}
__device__ __forceinline__ void store8(float* row, int c, int cols, bool on, const float* f) {
  const bool odd = (c & 8) != 0;
  float4 o;
  o.x = __shfl_xor_sync(0xffffffffu, odd ? f[0] : f[4], 1);
  o.y = __shfl_xor_sync(0xffffffffu, odd ? f[1] : f[5], 1);
  o.z = __shfl_xor_sync(0xffffffffu, odd ? f[2] : f[6], 1);
  o.w = __shfl_xor_sync(0xffffffffu, odd ? f[3] : f[7], 1);
  const float4 lo = make_float4(f[0], f[1], f[2], f[3]), hi = make_float4(f[4], f[5], f[6], f[7]);
  // even: own first half, the neighbour's first half; odd: the neighbour's second half, own second half
  const int c0 = odd ? c - 4 : c, c1 = odd ? c + 4 : c + 8;
  if (on && c0 < cols) __stcs(reinterpret_cast<float4*>(row + c0), odd ? o : lo);
  if (on && c1 < cols) __stcs(reinterpret_cast<float4*>(row + c1), odd ? hi : o);
}

// The exponent field of the largest magnitude of a thread's 8 values.  bf16:
// on packed pairs (a NaN wins and has exponent 255, as an infinity has).
__device__ __forceinline__ uint32_t top8(const Vec8<__nv_bfloat16>& v, const float*) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v.a);
  const __nv_bfloat162 m =
      __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
  return max((b >> 7) & 0xffu, (b >> 23) & 0xffu);
}
__device__ __forceinline__ uint32_t top8(const Vec8<float>&, const float* f) {
  float m = 0.0f;  // max.NaN: a NaN wins
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(f[i])));
  return (__float_as_uint(m) >> 23) & 0xffu;
}

__device__ __forceinline__ uint32_t pack4(const uint32_t* b) {
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}
// q of 8 values and the exponent byte of their block (the four threads of a
// block exchange theirs; every lane of the warp takes part).  One fused
// multiply-add scales a value and rounds it to an integer: adding 1.5 2^23
// leaves the integer in the last mantissa bits (the conversion instructions
// run at an eighth of the rate).  What that does not cover is done once more
// the long way: a value that rounds to +-128 and takes the clamp (its byte is
// 0x80, which no other gives), a block whose scale is no fp32 number (e < 6)
// and one that is not finite.
template <typename T>
__device__ __forceinline__ uint2 keep8(const Vec8<T>& v, const float* f, uint32_t& e) {
  uint32_t m = top8(v, f);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  e = m;
  const float scale = __uint_as_float((260u - e) << 23);
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(f[i], scale, 12582912.0f));
  uint2 k = make_uint2(pack4(b), pack4(b + 4));
  const uint32_t x = k.x ^ 0x80808080u, y = k.y ^ 0x80808080u;  // a zero byte where q is 0x80
  const uint32_t clamped = (((x - 0x01010101u) & ~x) | ((y - 0x01010101u) & ~y)) & 0x80808080u;
  if (clamped != 0u || e - 6u > 248u) {
    const float inv = ckpt_inv_scale(e);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = __float_as_uint(fmaf(fminf(fmaxf(f[i] * inv, -127.0f / 64.0f), 127.0f / 64.0f), 64.0f, 12582912.0f));
    k = e == 255u ? make_uint2(0u, 0u) : make_uint2(pack4(b), pack4(b + 4));
  }
  return k;
}
// And back: the byte q + 128 under the exponent of 2^23 is 2^23 + 128 + q.
__device__ __forceinline__ void read8(const uint2& q, uint32_t e, float* f) {
  const F2 s = f2(ckpt_scale(e));
  const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
  auto byte = [&](int i) { return __uint_as_float(__byte_perm(w[i >> 2], 0x4B000000u, 0x7440 + (i & 3))); };
#pragma unroll
  for (int i = 0; i < 8; i += 2) un2((f2(byte(i), byte(i + 1)) + f2(-8388736.0f)) * s, f[i], f[i + 1]);
}


template <typename T>
__global__ void __launch_bounds__(256, 4) ckpt_quantize_vec_kernel(const T* __restrict__ src, const int32_t* n_rows,
                                                                int rows, int cols, int nb, int lx,
                                                                int8_t* __restrict__ q, uint8_t* __restrict__ e) {
  constexpr int kU = 4;
  const int tx = 1 << lx, x = threadIdx.x & (tx - 1), ny = 256 >> lx;
  const int n = live_rows(n_rows, rows);
  const Vec8<T> none = {};
  for (long long r0 = static_cast<long long>(blockIdx.x) * ny; r0 < n; r0 += static_cast<long long>(gridDim.x) * ny) {
    const long long r = r0 + (threadIdx.x >> lx);
    for (int c0 = 8 * x; c0 - 8 * x < cols; c0 += kU * 8 * tx) {
      Vec8<T> v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int c = c0 + u * 8 * tx;
        v[u] = r < n && c < cols ? load8(src + r * cols + c) : none;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int c = c0 + u * 8 * tx;
        if (c - 8 * x >= cols) break;  // behind the row for every lane
        float f[8];
        unpack8(v[u], f);
        uint32_t ex;
        const uint2 k = keep8(v[u], f, ex);
        if (r < n && c < cols) {
          *reinterpret_cast<uint2*>(q + r * cols + c) = k;
          if ((x & 3) == 0) e[r * nb + c / kBlk] = static_cast<uint8_t>(ex);
        }
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256, 4) ckpt_dequantize_vec_kernel(const int8_t* __restrict__ q,
                                                                  const uint8_t* __restrict__ e,
                                                                  const int32_t* __restrict__ row_index,
                                                                  const int32_t* n_rows, int rows, int src_rows,
                                                                  int cols, int nb, int lx, T* __restrict__ dst,
                                                                  int* status) {
  constexpr int kD = 4;
  const int tx = 1 << lx, x = threadIdx.x & (tx - 1), ny = 256 >> lx;
  const int n = live_rows(n_rows, rows);
  for (long long r0 = static_cast<long long>(blockIdx.x) * ny; r0 < n; r0 += static_cast<long long>(gridDim.x) * ny) {
    const long long r = r0 + (threadIdx.x >> lx);
    const bool live = r < n;
    const long long sr = !live ? -1 : row_index != nullptr ? row_index[r] : r;
    const bool ok = sr >= 0 && sr < src_rows;
    if (live && !ok && x == 0) set_status(status, MOE_DEVERR_BAD_ROW_TOKEN);
    for (int c0 = 8 * x; c0 - 8 * x < cols; c0 += kD * 8 * tx) {
      uint2 k[kD];
      uint32_t ex[kD];
#pragma unroll
      for (int u = 0; u < kD; ++u) {
        const int c = c0 + u * 8 * tx;
        const bool on = ok && c < cols;
        k[u] = on ? *reinterpret_cast<const uint2*>(q + sr * cols + c) : make_uint2(0u, 0u);
        ex[u] = on ? e[sr * nb + c / kBlk] : 0u;
      }
#pragma unroll
      for (int u = 0; u < kD; ++u) {
        const int c = c0 + u * 8 * tx;
        if (c - 8 * x >= cols) break;
        float f[8];
        read8(k[u], ex[u], f);
        store8(dst + r * cols, c, cols, live, f);
      }
    }
  }
}

template <typename TS, typename TD, bool SWIGLU>
__global__ void __launch_bounds__(256, 4) act_save_vec_kernel(const TS* __restrict__ h, const int32_t* n_rows, int rows,
                                                           int I, int nb, int lx, TD* __restrict__ a,
                                                           int8_t* __restrict__ q, uint8_t* __restrict__ e) {
  constexpr int H = SWIGLU ? 2 : 1, kU = SWIGLU ? 2 : 4;
  const int tx = 1 << lx, x = threadIdx.x & (tx - 1), ny = 256 >> lx;
  const int n = live_rows(n_rows, rows);
  const Vec8<TS> none = {};
  for (long long r0 = static_cast<long long>(blockIdx.x) * ny; r0 < n; r0 += static_cast<long long>(gridDim.x) * ny) {
    const long long r = r0 + (threadIdx.x >> lx);
    for (int c0 = 8 * x; c0 - 8 * x < I; c0 += kU * 8 * tx) {
      Vec8<TS> v[kU][H];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int c = c0 + u * 8 * tx;
#pragma unroll
        for (int j = 0; j < H; ++j) v[u][j] = r < n && c < I ? load8(h + (r * H + j) * I + c) : none;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int c = c0 + u * 8 * tx;
        if (c - 8 * x >= I) break;
        const bool on = r < n && c < I;
        float f[H][8], o[8];
#pragma unroll
        for (int j = 0; j < H; ++j) {
          unpack8(v[u][j], f[j]);
          uint32_t ex;
          const uint2 k = keep8(v[u][j], f[j], ex);
          if (on) {
            *reinterpret_cast<uint2*>(q + (r * H + j) * I + c) = k;
            if ((x & 3) == 0) e[(r * H + j) * nb + c / kBlk] = static_cast<uint8_t>(ex);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const F2 h0 = f2(f[0][i], f[0][i + 1]);
          if constexpr (SWIGLU) un2(swiglu(h0, f2(f[H - 1][i], f[H - 1][i + 1])), o[i], o[i + 1]);
          else un2(gelu_sig(h0), o[i], o[i + 1]);
        }
        store8(a + r * I, c, I, r < n, o);
      }
    }
  }
}

template <typename TS, typename TD, bool SWIGLU>
__global__ void __launch_bounds__(256, 4) act_backward_vec_kernel(const int8_t* __restrict__ q,
                                                               const uint8_t* __restrict__ e,
                                                               const TS* __restrict__ da,
                                                               const float* __restrict__ row_w, const int32_t* n_rows,
                                                               int rows, int I, int nb, int lx, TD* __restrict__ dh,
                                                               TD* __restrict__ wa, float* __restrict__ dw) {
  constexpr int H = SWIGLU ? 2 : 1, kU = SWIGLU ? 2 : 4;
  __shared__ float s_part[8];
  const int tx = 1 << lx, x = threadIdx.x & (tx - 1), ny = 256 >> lx;
  const int n = live_rows(n_rows, rows);
  const Vec8<TS> none = {};
  for (long long r0 = static_cast<long long>(blockIdx.x) * ny; r0 < n; r0 += static_cast<long long>(gridDim.x) * ny) {
    const long long r = r0 + (threadIdx.x >> lx);
    const bool live = r < n;
    const F2 w2 = f2(live && row_w != nullptr ? row_w[r] : 1.0f);
    F2 dot2 = f2(0.0f);
    for (int c0 = 8 * x; c0 - 8 * x < I; c0 += kU * 8 * tx) {
      uint2 k[kU][H];
      uint32_t ex[kU][H];
      Vec8<TS> v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int c = c0 + u * 8 * tx;
        const bool on = live && c < I;
        v[u] = on ? load8(da + r * I + c) : none;
#pragma unroll
        for (int j = 0; j < H; ++j) {
          k[u][j] = on ? *reinterpret_cast<const uint2*>(q + (r * H + j) * I + c) : make_uint2(0u, 0u);
          ex[u][j] = on ? e[(r * H + j) * nb + c / kBlk] : 0u;
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int c = c0 + u * 8 * tx;
        if (c - 8 * x >= I) break;
        float g[8], f[H][8], d[H][8], o[8];
        unpack8(v[u], g);
#pragma unroll
        for (int j = 0; j < H; ++j) read8(k[u][j], ex[u][j], f[j]);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const F2 h0 = f2(f[0][i], f[0][i + 1]), gi = f2(g[i], g[i + 1]);
          F2 act, di[2];
          if constexpr (SWIGLU) swiglu_grad(h0, f2(f[H - 1][i], f[H - 1][i + 1]), act, di[0], di[1]);
          else gelu_sig_grad(h0, act, di[0]);
          dot2 = fma2(gi, act, dot2);
          un2(w2 * act, o[i], o[i + 1]);
          const F2 wg = w2 * gi;
#pragma unroll
          for (int j = 0; j < H; ++j) un2(di[j] * wg, d[j][i], d[j][i + 1]);
        }
#pragma unroll
        for (int j = 0; j < H; ++j) store8(dh + (r * H + j) * I, c, I, live, d[j]);
        if (wa != nullptr) store8(wa + r * I, c, I, live, o);
      }
    }
    if (dw != nullptr) {
      // a row's threads are one aligned part of a warp, or whole warps: the
      // sum runs over the part, then over the warps in order
      float dot, dot1;
      un2(dot2, dot, dot1);
      dot += dot1;
      for (int o = min(tx, 32) >> 1; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (tx > 32) {
        if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (x == 0) {
          dot = 0.0f;
          for (int i = 0; i < (tx >> 5); ++i) dot += s_part[(threadIdx.x >> 5) + i];
        }
        __syncthreads();
      }
      if (x == 0 && live) dw[r] = dot;
    }
  }
}

// Threads along a row (as a power of two) and the grid.  As few as one warp a
// row where that makes 3 blocks an SM (long runs per thread, no block-wide
// reduction for dw), more where there are fewer rows (2000 x 4096 read back:
// 64 threads 10.3 us, 32 13.3, 128 12.3), and more in wide rows as long as a
// thread's run stays eight steps in whole batches of four: the block's rows
// lie closer together (GELU backward of 4097 x 8192: 128 threads 49 us, 32
// 53, 256 50; of 8192 x 16384: 256 threads 159, 32 173).  A backward without
// `wa` (`lean`) has a stream less to write and does better on one-warp rows
// (16384 x 8192: 149 us, 160 with 128 threads), from 6 blocks an SM on (4097
// x 8192: 64 threads 39, 32 43).  Of those the most that leave at most an
// eighth of them idle in the row's last step (192 columns: 8 threads three
// times, not 32 of which 8 idle).
struct Shape { int lx, grid; };
inline Shape shape(int rows, int cols, bool lean = false) {
  const int vecs = cols / 8;
  int lx = 5;
  while (lx < 8 && static_cast<long long>(rows) << lx < (lean ? 6ll : 3ll) * 256 * num_sms()) ++lx;
  while (!lean && lx < 8 && vecs >= 16 << lx && vecs % (8 << lx) == 0) ++lx;
  for (; lx > 2; --lx) {
    const int tx = 1 << lx, padded = (vecs + tx - 1) / tx * tx;
    if ((padded - vecs) * 8 <= padded) break;
  }
  const int ny = 256 >> lx;
  return {lx, std::min((rows - 1) / ny + 1, 32 * num_sms())};
}
inline bool vec_ok(int cols, const void* a, const void* b, const void* c, const void* d) {
  const uintptr_t any = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                        reinterpret_cast<uintptr_t>(c) | reinterpret_cast<uintptr_t>(d);
  return cols % 8 == 0 && any % 16 == 0;
}

inline int blocks_of(int cols) { return (cols + kBlk - 1) / kBlk; }
// A warp per piece of kB blocks of a row.
inline int warp_grid(int rows, int nb) {
  const long long units = static_cast<long long>(rows) * ((nb + kB - 1) / kB);
  return static_cast<int>(std::max<long long>(1, std::min<long long>((units + 7) / 8, 32ll * num_sms())));
}

}  // namespace

cudaError_t launch_ckpt_quantize(int dtype, const void* src, const int32_t* n_rows, int rows, int cols, int8_t* q,
                                 uint8_t* e, cudaStream_t s) {
  const int nb = blocks_of(cols), grid = warp_grid(rows, nb);
  if (vec_ok(cols, src, q, nullptr, nullptr)) {
    const Shape p = shape(rows, cols);
    if (dtype == MOE_DTYPE_BF16)
      ckpt_quantize_vec_kernel<<<p.grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(src), n_rows, rows, cols, nb,
                                                      p.lx, q, e);
    else
      ckpt_quantize_vec_kernel<<<p.grid, 256, 0, s>>>(static_cast<const float*>(src), n_rows, rows, cols, nb, p.lx, q,
                                                      e);
    return cudaGetLastError();
  }
  if (dtype == MOE_DTYPE_BF16)
    ckpt_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(src), n_rows, rows, cols, nb, q, e);
  else
    ckpt_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(src), n_rows, rows, cols, nb, q, e);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_dequantize(int dtype, const int8_t* q, const uint8_t* e, const int32_t* row_index,
                                   const int32_t* n_rows, int rows, int src_rows, int cols, void* dst, int* status,
                                   cudaStream_t s) {
  const int nb = blocks_of(cols), grid = warp_grid(rows, nb);
  if (vec_ok(cols, dst, q, nullptr, nullptr)) {
    const Shape p = shape(rows, cols);
    if (dtype == MOE_DTYPE_BF16)
      ckpt_dequantize_vec_kernel<<<p.grid, 256, 0, s>>>(q, e, row_index, n_rows, rows, src_rows, cols, nb, p.lx,
                                                        static_cast<__nv_bfloat16*>(dst), status);
    else
      ckpt_dequantize_vec_kernel<<<p.grid, 256, 0, s>>>(q, e, row_index, n_rows, rows, src_rows, cols, nb, p.lx,
                                                        static_cast<float*>(dst), status);
    return cudaGetLastError();
  }
  if (dtype == MOE_DTYPE_BF16)
    ckpt_dequantize_kernel<<<grid, 256, 0, s>>>(q, e, row_index, n_rows, rows, src_rows, cols, nb,
                                                static_cast<__nv_bfloat16*>(dst), status);
  else
    ckpt_dequantize_kernel<<<grid, 256, 0, s>>>(q, e, row_index, n_rows, rows, src_rows, cols, nb,
                                                static_cast<float*>(dst), status);
  return cudaGetLastError();
}

namespace {

template <typename TS, typename TD, bool SW>
void run_save(const void* h, const int32_t* n_rows, int rows, int I, void* a, int8_t* q, uint8_t* e, cudaStream_t s) {
  const int nb = blocks_of(I);
  const TS* hp = static_cast<const TS*>(h);
  TD* ap = static_cast<TD*>(a);
  if (vec_ok(I, h, a, q, nullptr)) {
    const Shape p = shape(rows, I);
    act_save_vec_kernel<TS, TD, SW><<<p.grid, 256, 0, s>>>(hp, n_rows, rows, I, nb, p.lx, ap, q, e);
  } else {
    act_save_kernel<TS, TD, SW><<<warp_grid(rows, nb), 256, 0, s>>>(hp, n_rows, rows, I, nb,
                                                                                             ap, q, e);
  }
}
template <typename TS, typename TD>
void run_save(bool sw, const void* h, const int32_t* n_rows, int rows, int I, void* a, int8_t* q, uint8_t* e,
              cudaStream_t s) {
  if (sw) run_save<TS, TD, true>(h, n_rows, rows, I, a, q, e, s);
  else run_save<TS, TD, false>(h, n_rows, rows, I, a, q, e, s);
}

template <typename TS, typename TD, bool SW>
void run_backward(const int8_t* q, const uint8_t* e, const void* da, const float* row_w, const int32_t* n_rows,
                  int rows, int I, void* dh, void* wa, float* dw, cudaStream_t s) {
  const int nb = blocks_of(I);
  const TS* dp = static_cast<const TS*>(da);
  TD* hp = static_cast<TD*>(dh);
  TD* wp = static_cast<TD*>(wa);
  if (vec_ok(I, q, da, dh, wa)) {
    const Shape p = shape(rows, I, wa == nullptr);
    act_backward_vec_kernel<TS, TD, SW><<<p.grid, 256, 0, s>>>(q, e, dp, row_w, n_rows, rows, I, nb, p.lx, hp, wp, dw);
  } else {
    // one warp a row where that fills the GPU, else a block
    const int wpr = rows >= 6 * 8 * num_sms() ? 1 : 8, per = 8 / wpr;
    act_backward_kernel<TS, TD, SW><<<std::min((rows - 1) / per + 1, 32 * num_sms()), 256, 0, s>>>(
        q, e, dp, row_w, n_rows, rows, I, nb, wpr, hp, wp, dw);
  }
}
template <typename TS, typename TD>
void run_backward(bool sw, const int8_t* q, const uint8_t* e, const void* da, const float* row_w,
                  const int32_t* n_rows, int rows, int I, void* dh, void* wa, float* dw, cudaStream_t s) {
  if (sw) run_backward<TS, TD, true>(q, e, da, row_w, n_rows, rows, I, dh, wa, dw, s);
  else run_backward<TS, TD, false>(q, e, da, row_w, n_rows, rows, I, dh, wa, dw, s);
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
