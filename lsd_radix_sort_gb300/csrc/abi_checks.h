// Argument checks and the counted launch that the C ABI's files over rows of
// scores share.  Host code only.
#pragma once
#include <cstdint>

#include "../../include/lsdrs.h"
#include "kernels.h"

namespace lsdrs {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

inline int score_bytes(int type) { return type == RS_SCORE_F32 ? 4 : 2; }
inline bool known_type(int type) { return type >= RS_SCORE_F16 && type <= RS_SCORE_F32; }
inline bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
// a pointer that must be there, aligned to its element
inline bool given(const void* p, int bytes) { return p != nullptr && aligned(p, bytes); }

// rows x cols with a row stride, all addresses inside 63 bits
inline bool matrix_ok(int64_t rows, int64_t cols, int64_t stride, int bytes) {
  if (stride < cols) return false;
  return stride <= (int64_t(1) << 62) / bytes / (rows > 0 ? rows : 1);
}

// Bytes from the first element of a matrix to past its last.
inline uint64_t extent(int64_t rows, int64_t cols, int64_t stride, int bytes) {
  return rows == 0 ? 0 : (static_cast<uint64_t>(rows - 1) * stride + cols) * bytes;
}

inline bool apart(const void* a, uint64_t an, const void* b, uint64_t bn) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return !(x < y + bn && y < x + an);
}

// The gradient lies exactly over the scores or apart from them.
inline bool grad_ok(const void* scores, int64_t stride, void* grad, int64_t grad_stride, int64_t rows,
             int64_t cols, int type) {
  const int es = score_bytes(type);
  if (!given(grad, es) || !matrix_ok(rows, cols, grad_stride, es)) return false;
  if (grad == scores && grad_stride == stride) return true;
  return apart(scores, extent(rows, cols, stride, es), grad,
               extent(rows, cols, grad_stride, es));
}

template <class F>
rs_status enqueue(int kernel, uint64_t units, void* stream, F&& launch) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto call = [&](int* launched) { return launch(launched, s); };
  try {
    const cudaError_t e = counted_launch(
        kernel, units, s,
        [](void* ctx, int* launched) { return (*static_cast<decltype(call)*>(ctx))(launched); },
        &call);
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
  } catch (...) {  // the profiling log could not grow
    return RS_ERR_CUDA;
  }
}

}  // namespace lsdrs
