// Matrix products grouped by expert on the CUDA cores: the fp32 data type
// (the tensor cores have no full-fp32 multiply) and bf16 widths that TMA
// cannot address (rows that are no multiple of 16 bytes).  One kernel for
// the three products of a linear layer over ragged row segments:
//   forward   y[r, n]   = sum_k x[r, k]  W_g[n, k] (+ b_g[n])
//   dgrad     dx[r, k]  = sum_n dy[r, n] W_g[n, k]
//   wgrad     dW_g[n,k] = sum_r dy[r, n] x[r, k]     over g's rows, and with
//             it db_g[n] = sum_r dy[r, n]: the tiles of the first columns have
//             dy's slices in shared memory, and each of their 16 threads of a
//             row block adds up one of a slice's 16 steps
// 64 x 64 output tiles, 16-deep slices through shared memory (fp32: four
// stages of 4-byte asynchronous copies, which suit any width and alignment;
// bf16: the next slice through registers), a 4 x 4 block of neighbouring sums per
// thread: two 16-byte shared loads feed 16 multiply-adds.  Every 128 terms the
// block's partial sums (the bias gradient's too) are added to its totals, so
// that a sum of thousands of terms does not lose the small ones; all orders
// are fixed.  Bound by issue and latency, a correctness path beside
// the tensor cores: 30 experts x 50 rows x 390 x 380 in 33 us (14 TF/s).
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kTM = 64, kTN = 64, kTK = 16, kThreads = 256;
constexpr int kChunkSlices = 8;
constexpr int kStages = 4;

// 4 bytes global -> shared, or zeros (nothing is read then).
__device__ __forceinline__ void copy4_async(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
  float* db;    // wgrad: [G, M] column sums of A, or null
  int* status;  // cleared by the first block (nothing here sets it)
};

template <typename T, typename TO, bool WGRAD>
__global__ void __launch_bounds__(kThreads, 2) grouped_simt_kernel(const Args p) {
  constexpr bool kAsync = sizeof(T) == 4;
  __shared__ __align__(16) float As[kStages][kTK][kTM + 4];
  __shared__ __align__(16) float Bs[kStages][kTK][kTN + 4];
  __shared__ int s_off[kMaxExperts + 1];
  __shared__ int s_tstart[kMaxExperts + 1];
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
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
    const bool sums = WGRAD && p.db != nullptr && n0 == 0;
    // of the steps that are tx modulo 16, and their total of the chunks before
    float4 colsum = make_float4(0.f, 0.f, 0.f, 0.f), coltot = colsum;
    int slices = 0;
    // This thread's elements of a slice, along each operand's contiguous
    // index: four of A and four of B.  Their addresses in the first slice, and for each how many
    // contraction steps are left from there (0: a row or column behind the tile).
    constexpr int kPer = kTM * kTK / kThreads;
    const int tid = threadIdx.x;
    const T *pa[kPer], *pb[kPer];
    int left_a[kPer], left_b[kPer];
    int ma[kPer], ca[kPer], nb[kPer], db[kPer];
    const int len = static_cast<int>(c1 - c0);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid + j * kThreads;
      if (p.a_sc == 1) { ca[j] = i & (kTK - 1); ma[j] = i / kTK; } else { ma[j] = i & (kTM - 1); ca[j] = i / kTM; }
      if (p.b_sc == 1) { db[j] = i & (kTK - 1); nb[j] = i / kTK; } else { nb[j] = i & (kTN - 1); db[j] = i / kTN; }
      left_a[j] = ma[j] < nm ? len - ca[j] : 0;
      left_b[j] = n0 + nb[j] < p.N ? len - db[j] : 0;
      pa[j] = left_a[j] > 0 ? A + (m0 + ma[j]) * p.a_sm + (c0 + ca[j]) * p.a_sc : A;
      pb[j] = left_b[j] > 0 ? B + bg + (n0 + nb[j]) * p.b_sn + (c0 + db[j]) * p.b_sc : B;
    }
    const long long step_a = kTK * p.a_sc, step_b = kTK * p.b_sc;
    int at_k = 0;  // contraction steps of the slices asked for so far
    float ra[kPer], rb[kPer];
    auto copy = [&](int to) {  // fp32: the next slice into stage `to`, asynchronously
      if constexpr (kAsync) {
        if (at_k < len) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const bool oka = at_k < left_a[j], okb = at_k < left_b[j];
            copy4_async(&As[to][ca[j]][ma[j]], oka ? pa[j] : A, oka);
            copy4_async(&Bs[to][db[j]][nb[j]], okb ? pb[j] : B, okb);
            pa[j] += step_a;
            pb[j] += step_b;
          }
        }
        at_k += kTK;
        copies_commit();  // an empty group behind the end keeps the count
      }
    };
    auto fetch = [&]() {  // bf16: the next slice into registers
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        ra[j] = at_k < left_a[j] ? to_f32(*pa[j]) : 0.f;
        rb[j] = at_k < left_b[j] ? to_f32(*pb[j]) : 0.f;
        pa[j] += step_a;
        pb[j] += step_b;
      }
      at_k += kTK;
    };
    auto put = [&](int to) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        As[to][ca[j]][ma[j]] = ra[j];
        Bs[to][db[j]][nb[j]] = rb[j];
      }
    };
    int st = 0;
    if constexpr (kAsync) {
      for (int i = 0; i < kStages - 1; ++i) copy(i);
    } else if (len > 0) {
      fetch();
    }
    for (int k0 = 0; k0 < len; k0 += kTK, st = (st + 1) & (kStages - 1)) {
      if constexpr (kAsync) {
        copies_wait<kStages - 2>();  // this slice has arrived (for this thread)
        __syncthreads();             // for every thread, and the stage before is read
        copy((st + kStages - 1) & (kStages - 1));
      } else {
        put(st);
        __syncthreads();
        if (k0 + kTK < len) fetch();
      }
#pragma unroll
      for (int kk = 0; kk < kTK; ++kk) {
        const float4 a4 = *reinterpret_cast<const float4*>(&As[st][kk][4 * ty]);
        const float4 b4 = *reinterpret_cast<const float4*>(&Bs[st][kk][4 * tx]);
        const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
      }
      if (WGRAD && sums) {
        const float4 v = *reinterpret_cast<const float4*>(&As[st][tx][4 * ty]);
        colsum.x += v.x; colsum.y += v.y; colsum.z += v.z; colsum.w += v.w;
      }
      if (++slices == kChunkSlices) {
        slices = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) { tot[i][j] += acc[i][j]; acc[i][j] = 0.f; }
        if (WGRAD && sums) {
          coltot.x += colsum.x; coltot.y += colsum.y; coltot.z += colsum.z; coltot.w += colsum.w;
          colsum = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
    if constexpr (kAsync) copies_wait<0>();
    __syncthreads();  // the tile's stages are read before the next tile fills them
    if (WGRAD && sums) {
      float v[4] = {coltot.x + colsum.x, coltot.y + colsum.y, coltot.z + colsum.z, coltot.w + colsum.w};
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      float* out = p.db + static_cast<long long>(g) * p.M + m0 + 4 * ty;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (tx == 0 && 4 * ty + i < nm) out[i] = p.accumulate ? out[i] + v[i] : v[i];
    }
    const long long cg = WGRAD ? static_cast<long long>(g) * p.c_gstride : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = 4 * ty + i;
      if (m >= nm) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + 4 * tx + j;
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

template <typename T, typename TO, bool WGRAD>
cudaError_t run(const Args& a, long long tiles, cudaStream_t s) {
  const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(tiles, 6ll * num_sms())));
  grouped_simt_kernel<T, TO, WGRAD><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedLaunch& L, int* status, cudaStream_t s) {
  Args a = {};
  a.status = status;
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
    a.db = L.db;
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

}  // namespace moe
