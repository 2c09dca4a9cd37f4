// Matrix products grouped by expert on the CUDA cores: the fp32 data type
// (the tensor cores have no full-fp32 multiply) and bf16 widths that TMA
// cannot address (rows that are no multiple of 16 bytes).  One kernel for
// the three products of a linear layer over ragged row segments:
//   forward   y[r, n]   = sum_k x[r, k]  W_g[n, k] (+ b_g[n])
//   dgrad     dx[r, k]  = sum_n dy[r, n] W_g[n, k]
//   wgrad     dW_g[n,k] = sum_r dy[r, n] x[r, k]     over g's rows
// 64 x 64 output tiles, 16-deep slices through shared memory, a 4 x 4 block
// of sums per thread.  Every 128 terms the block's partial sums are added to
// its totals, so that a sum of thousands of terms does not lose the small
// ones; all orders are fixed.
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kTM = 64, kTN = 64, kTK = 16, kThreads = 256;
constexpr int kChunkSlices = 8;

struct Args {
  const void* A; long long a_sm, a_sc;             // A(m, c) = A[m a_sm + c a_sc]
  const void* B; long long b_sn, b_sc, b_gstride;  // B(n, c) = B[g b_gstride + n b_sn + c b_sc]
  const void* bias;                                // [G, n] or null (forward)
  void* C; long long ldc, c_gstride;
  const int32_t* offsets;
  int G, rows;
  int M;        // wgrad: output rows per group
  int N;        // output columns
  int Kc;       // contraction length (forward, dgrad)
  int col_tiles;
  int accumulate;
};

template <typename T, typename TO, bool WGRAD>
__global__ void __launch_bounds__(kThreads) grouped_simt_kernel(const Args p) {
  __shared__ float As[kTK][kTM + 1];
  __shared__ float Bs[kTK][kTN + 1];
  __shared__ int s_off[kMaxExperts + 1];
  __shared__ int s_tstart[kMaxExperts + 1];
  const T* A = static_cast<const T*>(p.A);
  const T* B = static_cast<const T*>(p.B);
  const int G = p.G;
  // segment bounds inside [0, rows]; a segment that ends before it starts is empty
  for (int i = threadIdx.x; i <= G; i += kThreads) s_off[i] = max(0, min(p.offsets[i], p.rows));
  __syncthreads();
  const int m_tiles_w = (p.M + kTM - 1) / kTM;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int base = 0; base < G; base += 32) {
      const int g = base + lane;
      int v = 0;
      if (g < G) v = (WGRAD ? m_tiles_w : (max(0, s_off[g + 1] - s_off[g]) + kTM - 1) / kTM) * p.col_tiles;
      int incl = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += t;
      }
      if (g < G) s_tstart[g] = carry + incl - v;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_tstart[G] = carry;
  }
  __syncthreads();
  const int total = s_tstart[G];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_tstart[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    const int g = lo, local = tile - s_tstart[g];
    const int mt = local / p.col_tiles, n0 = (local - mt * p.col_tiles) * kTN;
    const int seg0 = s_off[g], seg1 = max(s_off[g], s_off[g + 1]);
    const long long m0 = WGRAD ? static_cast<long long>(mt) * kTM : static_cast<long long>(seg0) + mt * kTM;
    const int nm = WGRAD ? min(kTM, p.M - mt * kTM) : min(kTM, seg1 - seg0 - mt * kTM);
    const long long c0 = WGRAD ? seg0 : 0, c1 = WGRAD ? seg1 : p.Kc;
    const long long bg = static_cast<long long>(g) * p.b_gstride;
    float acc[4][4] = {}, tot[4][4] = {};
    int slices = 0;
    for (long long k0 = c0; k0 < c1; k0 += kTK) {
      for (int i = threadIdx.x; i < kTM * kTK; i += kThreads) {
        // neighbouring threads read along each operand's contiguous index
        int m, c;
        if (p.a_sc == 1) { c = i & (kTK - 1); m = i / kTK; } else { m = i & (kTM - 1); c = i / kTM; }
        As[c][m] = (m < nm && k0 + c < c1) ? to_f32(A[(m0 + m) * p.a_sm + (k0 + c) * p.a_sc]) : 0.f;
        int n, d;
        if (p.b_sc == 1) { d = i & (kTK - 1); n = i / kTK; } else { n = i & (kTN - 1); d = i / kTN; }
        Bs[d][n] = (n0 + n < p.N && k0 + d < c1) ? to_f32(B[bg + (n0 + n) * p.b_sn + (k0 + d) * p.b_sc]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kTK; ++kk) {
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = As[kk][ty + 16 * i];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = Bs[kk][tx + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
      }
      if (++slices == kChunkSlices) {
        slices = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) { tot[i][j] += acc[i][j]; acc[i][j] = 0.f; }
      }
      __syncthreads();
    }
    const long long cg = WGRAD ? static_cast<long long>(g) * p.c_gstride : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = ty + 16 * i;
      if (m >= nm) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 16 * j;
        if (n >= p.N) continue;
        float v = tot[i][j] + acc[i][j];
        if (p.bias != nullptr) v += to_f32(static_cast<const T*>(p.bias)[static_cast<long long>(g) * p.N + n]);
        TO* dst = static_cast<TO*>(p.C) + cg + (m0 + m) * p.ldc + n;
        if (WGRAD && p.accumulate) v += to_f32(*dst);
        *dst = from_f32<TO>(v);
      }
    }
  }
}

// db[g, n] (+)= sum over g's rows of dy[r, n].  A block takes `share` of the
// segment's rows (blockIdx.z) for 64 columns: its eight warps take every
// eighth row, two columns a thread and eight rows in flight, and their sums
// are added in warp order.  With more than one share the blocks leave partial
// sums [share][G][N], which grouped_colsum_join_kernel adds in order.  Bound
// by reading dy once.
template <typename T>
__device__ __forceinline__ float2 ld2(const T* p, bool second);
template <>
__device__ __forceinline__ float2 ld2(const float* p, bool second) {
  return make_float2(p[0], second ? p[1] : 0.f);
}
template <>
__device__ __forceinline__ float2 ld2(const __nv_bfloat16* p, bool second) {
  return make_float2(__bfloat162float(p[0]), second ? __bfloat162float(p[1]) : 0.f);
}

template <typename T, bool PAIRED>
__global__ void __launch_bounds__(256) grouped_colsum_kernel(const T* __restrict__ dy,
                                                             const int32_t* __restrict__ offsets, int rows, int N,
                                                             int accumulate, float* __restrict__ out) {
  __shared__ float2 s[8][32];
  const int g = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = max(0, min(offsets[g], rows)), e = max(b, max(0, min(offsets[g + 1], rows)));
  const int per = (e - b + gridDim.z - 1) / gridDim.z;
  const int r0 = min(e, b + static_cast<int>(blockIdx.z) * per), r1 = min(e, r0 + per);
  const int n = blockIdx.x * 64 + 2 * lane;
  float2 a = make_float2(0.f, 0.f);
  if (n < N) {
    const bool two = n + 1 < N;
    const T* p = dy + static_cast<long long>(r0 + warp) * N + n;
    const long long step = 8ll * N;
    int r = r0 + warp;
    for (; r + 56 < r1; r += 64, p += 8 * step) {
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (PAIRED) {  // N is even and dy on a whole pair: one load for both columns
          if constexpr (sizeof(T) == 2)
            v[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p + i * step));
          else
            v[i] = *reinterpret_cast<const float2*>(p + i * step);
        } else {
          v[i] = ld2(p + i * step, two);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) { a.x += v[i].x; a.y += v[i].y; }
    }
    for (; r < r1; r += 8, p += step) {
      const float2 v = ld2(p, two);
      a.x += v.x;
      a.y += v.y;
    }
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && n < N) {
    float2 v = s[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) { v.x += s[i][lane].x; v.y += s[i][lane].y; }
    float* o = out + (static_cast<long long>(blockIdx.z) * gridDim.y + g) * N + n;
    o[0] = accumulate ? o[0] + v.x : v.x;
    if (n + 1 < N) o[1] = accumulate ? o[1] + v.y : v.y;
  }
}

__global__ void __launch_bounds__(256) grouped_colsum_join_kernel(const float* __restrict__ part, int shares,
                                                                  long long n, int accumulate,
                                                                  float* __restrict__ db) {
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    float v = accumulate ? db[i] : 0.f;
    for (int z = 0; z < shares; ++z) v += part[z * n + i];
    db[i] = v;
  }
}

template <typename T, typename TO, bool WGRAD>
cudaError_t run(const Args& a, long long tiles, cudaStream_t s) {
  const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(tiles, 6ll * num_sms())));
  grouped_simt_kernel<T, TO, WGRAD><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedLaunch& L, cudaStream_t s) {
  Args a = {};
  a.offsets = L.offsets;
  a.G = L.G;
  a.rows = L.rows;
  const long long NK = static_cast<long long>(L.N) * L.K;
  if (L.dir == kGroupedWgrad) {
    a.A = L.dy; a.a_sm = 1; a.a_sc = L.N;
    a.B = L.x; a.b_sn = 1; a.b_sc = L.K; a.b_gstride = 0;
    a.C = L.out; a.ldc = L.K; a.c_gstride = NK;
    a.M = L.N; a.N = L.K;
    a.accumulate = L.accumulate;
  } else if (L.dir == kGroupedDgrad) {
    a.A = L.dy; a.a_sm = L.N; a.a_sc = 1;
    a.B = L.w; a.b_sn = 1; a.b_sc = L.K; a.b_gstride = NK;
    a.C = L.out; a.ldc = L.K;
    a.N = L.K; a.Kc = L.N;
  } else {
    a.A = L.x; a.a_sm = L.K; a.a_sc = 1;
    a.B = L.w; a.b_sn = L.K; a.b_sc = 1; a.b_gstride = NK;
    a.C = L.out; a.ldc = L.N;
    a.N = L.N; a.Kc = L.K;
    a.bias = L.bias;
  }
  a.col_tiles = (a.N + kTN - 1) / kTN;
  const bool bf = L.dtype == MOE_DTYPE_BF16, obf = L.out_dtype == MOE_DTYPE_BF16;
  if (L.dir == kGroupedWgrad) {
    const long long tiles = static_cast<long long>(L.G) * ((a.M + kTM - 1) / kTM) * a.col_tiles;
    return bf ? run<__nv_bfloat16, float, true>(a, tiles, s) : run<float, float, true>(a, tiles, s);
  }
  const long long tiles = (L.rows / kTM + std::min<long long>(L.G, L.rows)) * a.col_tiles;
  if (bf) return obf ? run<__nv_bfloat16, __nv_bfloat16, false>(a, tiles, s) : run<__nv_bfloat16, float, false>(a, tiles, s);
  return run<float, float, false>(a, tiles, s);
}

int grouped_colsum_shares(int G, int rows, int N) {
  const long long blocks = static_cast<long long>((N + 63) / 64) * G;
  // eight blocks an SM, of 128 rows of an even segment at least
  const long long want = (8ll * 148 + blocks - 1) / blocks, most = (static_cast<long long>(rows) / G + 127) / 128;
  return static_cast<int>(std::max<long long>(1, std::min<long long>({want, most, 64})));
}

cudaError_t launch_grouped_colsum(int dtype, const void* dy, const int32_t* offsets, int G, int rows, int N,
                                  int accumulate, float* db, float* part, cudaStream_t s) {
  const int shares = grouped_colsum_shares(G, rows, N);
  const dim3 grid((N + 63) / 64, G, shares);
  float* out = shares > 1 ? part : db;
  const int acc = shares > 1 ? 0 : accumulate;
  const bool pair = N % 2 == 0 && reinterpret_cast<uintptr_t>(dy) % 8 == 0;
  if (dtype == MOE_DTYPE_BF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(dy);
    if (pair) grouped_colsum_kernel<__nv_bfloat16, true><<<grid, 256, 0, s>>>(p, offsets, rows, N, acc, out);
    else grouped_colsum_kernel<__nv_bfloat16, false><<<grid, 256, 0, s>>>(p, offsets, rows, N, acc, out);
  } else {
    const float* p = static_cast<const float*>(dy);
    if (pair) grouped_colsum_kernel<float, true><<<grid, 256, 0, s>>>(p, offsets, rows, N, acc, out);
    else grouped_colsum_kernel<float, false><<<grid, 256, 0, s>>>(p, offsets, rows, N, acc, out);
  }
  if (shares > 1) {
    const long long n = static_cast<long long>(G) * N;
    const int blocks = static_cast<int>(std::min<long long>((n + 255) / 256, 4ll * num_sms()));
    grouped_colsum_join_kernel<<<blocks, 256, 0, s>>>(part, shares, n, accumulate, db);
  }
  return cudaGetLastError();
}

}  // namespace moe
