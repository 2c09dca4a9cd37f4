// The column sums of a row segment, shared by the kernels that take them.
#pragma once

#include "common.cuh"

namespace moe {

// db[g, n] (+)= sum over g's rows of dy[r, n].  A block of 256 threads takes
// share `z` of `shares` of group g's rows for the 64 columns of column tile
// `nt`: its eight warps take every eighth row, two columns a thread and eight
// rows in flight, and their sums are added in warp order.  With more than one
// share the blocks leave partial sums, which a second kernel adds in order.
// Bound by reading dy once.
template <typename T>
__device__ __forceinline__ float2 ld2(const T* p, bool second) {
  return make_float2(to_f32(p[0]), second ? to_f32(p[1]) : 0.f);
}
// N even and p on a whole pair: one load for both columns
__device__ __forceinline__ float2 ld2_pair(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ld2_pair(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

// `out`: row g's N sums (or the share's partial ones); `s`: shared memory.
template <typename T, bool PAIRED>
__device__ __forceinline__ void grouped_colsum_block(const T* __restrict__ dy, const int32_t* __restrict__ offsets,
                                                     int rows, int N, int nt, int g, int z, int shares, int accumulate,
                                                     float* __restrict__ out, float2 (*s)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = max(0, min(offsets[g], rows)), e = max(b, max(0, min(offsets[g + 1], rows)));
  const int per = (e - b + shares - 1) / shares;
  const int r0 = static_cast<int>(min(static_cast<long long>(e), b + static_cast<long long>(z) * per));
  const int r1 = min(e, r0 + per);
  const int n = nt * 64 + 2 * lane;
  float2 a = make_float2(0.f, 0.f);
  if (n < N) {
    const bool two = n + 1 < N;
    const T* p = dy + static_cast<long long>(r0 + warp) * N + n;
    const long long step = 8ll * N;
    int r = r0 + warp;
    for (; r + 56 < r1; r += 64, p += 8 * step) {
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = PAIRED ? ld2_pair(p + i * step) : ld2(p + i * step, two);
#pragma unroll
      for (int i = 0; i < 8; ++i) { a.x += v[i].x; a.y += v[i].y; }
    }
    for (; r < r1; r += 8, p += step) {
      const float2 v = PAIRED ? ld2_pair(p) : ld2(p, two);
      a.x += v.x;
      a.y += v.y;
    }
  }
  __syncthreads();  // `s` of an earlier tile is read
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && n < N) {
    float2 v = s[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) { v.x += s[i][lane].x; v.y += s[i][lane].y; }
    out[n] = accumulate ? out[n] + v.x : v.x;
    if (n + 1 < N) out[n + 1] = accumulate ? out[n + 1] + v.y : v.y;
  }
}

}  // namespace moe
