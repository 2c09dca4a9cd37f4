// Host helpers shared by the files that implement the C ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kernels.cuh"

namespace moe {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Carves a caller's workspace into 256-byte aligned regions.
struct Carve {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off += align_up(bytes);
    return o;
  }
};

inline size_t esize(int dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }
inline bool is_dtype(int dtype) { return dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16; }

inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
#define MOE_TRY(expr)                          \
  do {                                         \
    moe_status_t st_ = (expr);                 \
    if (st_ != MOE_OK) return st_;             \
  } while (0)
#define MOE_CUDA(expr) MOE_TRY(cuda_status(expr))

inline bool aligned_ws(const void* ws) { return (reinterpret_cast<uintptr_t>(ws) % kAlign) == 0; }
// bf16 tensors that the tensor-core kernels move with TMA, and the fp32
// weight gradients they store with it, start on a 16-byte boundary.
inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename P> inline P at(void* ws, size_t off) {
  return reinterpret_cast<P>(static_cast<char*>(ws) + off);
}

}  // namespace moe
