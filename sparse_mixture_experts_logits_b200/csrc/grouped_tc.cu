// Matrix products grouped by expert on the tensor cores: bf16 operands whose
// rows are whole 16-byte units (N and K multiples of 8).  The three products
// are the three operand layouts of the tokens-on-N GEMM; this file gives each
// its launch, and prepares the ragged weight gradient.
//
// Measured, back to back under the power cap (990 W, 0.95 to 1.6 GHz), which
// is what bounds the large ones: 64 experts x 256 rows x 8192 x 2048 0.59 ms
// (930 TF/s; a cuBLAS batched product of the same size 0.62), the same with
// uneven segments 0.66, 8 x 2048 rows 0.45 ms (1210 TF/s; 0.42).  Weight
// gradients write N x K fp32 per expert: 32 x 512 rows x 2048 x 5120 in 0.42
// ms, 0.53 when added onto.  Few rows: 256 over 160 experts x 5120 x 1536 in
// 0.34 ms, 5.9 TB/s of weights.
#include <algorithm>

#include "gemm_sm100.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr size_t kHead = 256;  // status word and tile counters
constexpr int kTail = kBK;     // rows of a group's tail buffer: one k-block

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Rows [b, e) of group g; without offsets there is one group, of all rows.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ offsets, int g, int rows, int& b, int& e) {
  b = offsets != nullptr ? max(0, min(offsets[g], rows)) : 0;
  e = offsets != nullptr ? max(b, min(offsets[g + 1], rows)) : rows;
}

// db[g, n] (+)= sum over g's rows of dy[r, n] (N even).  A block of 256
// threads takes share `z` of `shares` of group g's rows for the 64 columns of
// column tile `nt`: its eight warps take every eighth row, two columns a
// thread and eight rows in flight, and their sums are added in warp order.  A
// thread's sum goes to its total every 128 rows, so that a long segment's does
// not lose the small ones.
// With more than one share the blocks leave partial sums, which a second
// kernel adds in order.  Bound by reading dy once.  `out`: group g's N sums
// (or the share's partial ones); `s`: shared memory.
__device__ __forceinline__ void colsum_block(const __nv_bfloat16* __restrict__ dy, const int32_t* __restrict__ offsets,
                                             int rows, int N, int nt, int g, int z, int shares, int accumulate,
                                             float* __restrict__ out, float2 (*s)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b, e;
  group_rows(offsets, g, rows, b, e);
  const int per = (e - b + shares - 1) / shares;
  const int r0 = static_cast<int>(min(static_cast<long long>(e), b + static_cast<long long>(z) * per));
  const int r1 = min(e, r0 + per);
  const int n = nt * 64 + 2 * lane;
  float2 a = make_float2(0.f, 0.f), tot = a;
  if (n < N) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(dy + static_cast<long long>(r0 + warp) * N + n);
    const long long step = 4ll * N;
    int r = r0 + warp, turns = 0;
    for (; r + 56 < r1; r += 64, p += 8 * step) {
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __bfloat1622float2(p[i * step]);
#pragma unroll
      for (int i = 0; i < 8; ++i) { a.x += v[i].x; a.y += v[i].y; }
      if (++turns == 16) {
        turns = 0;
        tot.x += a.x;
        tot.y += a.y;
        a = make_float2(0.f, 0.f);
      }
    }
    for (; r < r1; r += 8, p += step) {
      const float2 v = __bfloat1622float2(*p);
      a.x += v.x;
      a.y += v.y;
    }
  }
  __syncthreads();  // `s` of an earlier tile is read
  s[warp][lane] = make_float2(tot.x + a.x, tot.y + a.y);
  __syncthreads();
  if (warp == 0 && n < N) {
    float2 v = s[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) { v.x += s[i][lane].x; v.y += s[i][lane].y; }
    out[n] = accumulate ? out[n] + v.x : v.x;
    out[n + 1] = accumulate ? out[n + 1] + v.y : v.y;
  }
}

__global__ void __launch_bounds__(256) colsum_kernel(const __nv_bfloat16* __restrict__ dy,
                                                     const int32_t* __restrict__ offsets, int rows, int N,
                                                     int accumulate, float* __restrict__ out) {
  __shared__ float2 s[8][32];
  colsum_block(dy, offsets, rows, N, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z, accumulate,
               out + (static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y) * N, s);
}

__global__ void __launch_bounds__(256) colsum_join_kernel(const float* __restrict__ part, int shares, long long n,
                                                          int accumulate, float* __restrict__ db) {
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    float v = accumulate ? db[i] : 0.f;
    for (int z = 0; z < shares; ++z) v += part[z * n + i];
    db[i] = v;
  }
}

cudaError_t launch_colsum(const GroupedLaunch& L, cudaStream_t s) {
  const int shares = grouped_colsum_shares(L.G, L.rows, L.N);
  colsum_kernel<<<dim3((L.N + 63) / 64, L.G, shares), 256, 0, s>>>(
      static_cast<const __nv_bfloat16*>(L.dy), L.offsets, L.rows, L.N, shares > 1 ? 0 : L.accumulate,
      shares > 1 ? L.part : L.db);
  if (shares > 1) {
    const long long n = static_cast<long long>(L.G) * L.N;
    const int blocks = static_cast<int>(std::min<long long>((n + 255) / 256, 4ll * num_sms()));
    colsum_join_kernel<<<blocks, 256, 0, s>>>(L.part, shares, n, L.accumulate, L.db);
  }
  return cudaGetLastError();
}

// Before a ragged weight gradient.  For group g = blockIdx.y with rows
// [b, e): its last (e - b) % 64 rows of src, filled up with zero rows to 64,
// go to tail[g * 64 ..]; a group without rows gets its `out` zeroed unless it
// is added onto.  blockIdx.x shares the 16-byte units of each; blockIdx.z
// picks the operand.  Blocks of blockIdx.z = 2 take db's column sums when
// they are few (a launch saved), and the first block clears the status word.
__global__ void __launch_bounds__(256) wgrad_prepare_kernel(const uint4* __restrict__ x, const uint4* __restrict__ dy,
                                                            const int32_t* __restrict__ offsets, int rows, int vk,
                                                            int vn, long long out_units, int accumulate,
                                                            uint4* __restrict__ x_tail, uint4* __restrict__ dy_tail,
                                                            uint4* __restrict__ out, float* __restrict__ db,
                                                            int* status) {
  grid_launch_dependents();
  if (status != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *status = 0;
  const int g = blockIdx.y;
  if (blockIdx.z == 2) {
    __shared__ float2 part[8][32];
    for (int nt = blockIdx.x; nt * 64 < 8 * vn; nt += gridDim.x)
      colsum_block(reinterpret_cast<const __nv_bfloat16*>(dy), offsets, rows, 8 * vn, nt, g, 0, 1, accumulate,
                   db + static_cast<long long>(g) * 8 * vn, part);
    return;
  }
  int b, e;
  group_rows(offsets, g, rows, b, e);
  const int tid = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (e <= b) {
    if (accumulate) return;
    uint4* o = out + g * out_units;
    for (long long i = static_cast<long long>(blockIdx.z) * step + tid; i < out_units; i += 2ll * step) o[i] = zero;
    return;
  }
  const int t = (e - b) & (kTail - 1);
  if (t == 0) return;
  const int v = blockIdx.z ? vn : vk;
  const uint4* src = (blockIdx.z ? dy : x) + static_cast<long long>(e - t) * v;
  uint4* dst = (blockIdx.z ? dy_tail : x_tail) + static_cast<long long>(g) * kTail * v;
  for (int i = tid; i < kTail * v; i += step) dst[i] = i < t * v ? src[i] : zero;
}

}  // namespace

bool grouped_tc_ok(int dtype, int N, int K) { return dtype == MOE_DTYPE_BF16 && N % 8 == 0 && K % 8 == 0; }

int grouped_colsum_shares(int G, int rows, int N) {
  const long long blocks = static_cast<long long>((N + 63) / 64) * G;
  // eight blocks an SM, of 128 rows of an even segment at least
  const long long want = (8ll * 148 + blocks - 1) / blocks, most = (static_cast<long long>(rows) / G + 127) / 128;
  return static_cast<int>(std::max<long long>(1, std::min<long long>({want, most, 64})));
}

size_t grouped_tc_workspace(int dir, int G, int N, int K) {
  if (dir != kGroupedWgrad) return kHead;
  const size_t rows = static_cast<size_t>(G) * kTail * 2;
  return kHead + up256(rows * K) + up256(rows * N);
}

cudaError_t launch_grouped_tc(const GroupedLaunch& L, void* ws, cudaStream_t s) {
  char* base = static_cast<char*>(ws);
  const long long wrows = static_cast<long long>(L.G) * L.N;
  SwapLaunch S{};
  S.num_groups = L.G;
  S.offsets = L.offsets;
  S.rows = L.rows;
  S.status = L.status != nullptr ? L.status : reinterpret_cast<int*>(base);
  S.w_tile_step = 256; S.w_hi_offset = 64; S.w_cta_step = 128;
  S.cols_per_tile = 256;
  S.out = L.out;
  if (L.dir == kGroupedWgrad) {
    char* x_tail = base + kHead;
    char* dy_tail = x_tail + up256(static_cast<size_t>(L.G) * kTail * 2 * L.K);
    const int vk = L.K / 8, vn = L.N / 8;
    const long long units = static_cast<long long>(L.N) * L.K / 4;
    const long long most = std::max<long long>(kTail * static_cast<long long>(std::max(vk, vn)), units / 2);
    const int share = static_cast<int>(std::max<long long>(1, std::min<long long>((most + 1023) / 1024, 32)));
    // the sums beside the preparation when they are a wave of blocks at most (16384 x 8192: 76 us there, 51 apart)
    const bool sums = L.db != nullptr && grouped_colsum_shares(L.G, L.rows, L.N) == 1 &&
                      static_cast<long long>((L.N + 63) / 64) * L.G <= 4 * num_sms();
    wgrad_prepare_kernel<<<dim3(share, L.G, sums ? 3 : 2), 256, 0, s>>>(
        static_cast<const uint4*>(L.x), static_cast<const uint4*>(L.dy), L.offsets, L.rows, vk, vn, units,
        L.accumulate, reinterpret_cast<uint4*>(x_tail), reinterpret_cast<uint4*>(dy_tail), static_cast<uint4*>(L.out),
        L.db, L.status != nullptr ? nullptr : reinterpret_cast<int*>(base));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (L.db != nullptr && !sums) {
      e = launch_colsum(L, s);
      if (e != cudaSuccess) return e;
    }
    // A = x (the output's contiguous index), B = dy: dw[g][n][k]
    S.epi = EPI_OUT_F32;
    S.layout = kSwWgradRagged;
    S.W = L.x; S.w_rows = L.rows; S.a_cols = L.K;
    S.X = L.dy; S.x_rows = L.rows; S.b_cols = L.N;
    S.W_tail = x_tail; S.X_tail = dy_tail;
    S.w_tiles = (L.K + 255) / 256;
    S.b_tiles = (L.N + 255) / 256;
    S.out_cols = L.K; S.ldo = L.K;
    S.out_gstride = static_cast<long long>(L.N) * L.K;
    S.accumulate = L.accumulate;
    return launch_gemm_swap(S, s);
  }
  S.W = L.w; S.w_rows = wrows;
  // The tile counter balances what follows a CTA pair's first tile: a launch
  // that gives each pair one at most goes without it, and without the clear
  // of the counter (and of the status word) in a launch of its own.
  const int out_cols = L.dir == kGroupedDgrad ? L.K : L.N;
  const long long tiles = (L.rows / 256 + std::min(L.G, L.rows)) * static_cast<long long>((out_cols + 255) / 256);
  if (2 * tiles <= num_sms()) {
    S.clear_status = 1;
  } else {
    S.tile_ctr = reinterpret_cast<int*>(base) + 2;
    const cudaError_t e = cudaMemsetAsync(base, 0, 16, s);
    if (e != cudaSuccess) return e;
  }
  if (L.dir == kGroupedDgrad) {
    S.layout = kSwDgrad;
    S.X = L.dy; S.x_rows = L.rows;
    S.K = L.N;
    S.a_cols = L.K;
    S.out_cols = L.K; S.ldo = L.K;
  } else {
    S.layout = kSwFwd;
    S.X = L.x; S.x_rows = L.rows;
    S.K = L.K;
    S.w_rows_per_group = L.N;
    S.out_cols = L.N; S.ldo = L.N;
    S.bias = L.bias;
  }
  S.epi = L.out_dtype != MOE_DTYPE_BF16 ? EPI_OUT_F32 : S.K > kSwWholeBf16 ? EPI_OUT_BF16_CHUNKED : EPI_OUT_BF16;
  S.w_tiles = (S.out_cols + 255) / 256;
  return launch_gemm_swap(S, s);
}

}  // namespace moe
