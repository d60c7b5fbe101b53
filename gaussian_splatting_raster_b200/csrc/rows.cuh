// Shared by the per-row operators (lookup.cu, ffn*.cu): element types, argument checks and the
// status word of their bounded waits. These operators need no workspace: outputs and scratch are
// the caller's, so calls on different streams, or graphs captured with different scratch, never
// share memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "splat.h"

namespace splat {
namespace rows {

inline int elem_size(int dtype) {
  return dtype == SPLAT_F32 ? 4 : (dtype == SPLAT_BF16 || dtype == SPLAT_F16) ? 2 : 0;
}

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_f<__half>(float v) {
  return __float2half_rn(v);
}

// One row-strided array argument: `rows` rows of `cols` elements of `elem` bytes, `ld` elements
// apart. Absent (NULL) arrays are given rows = 0.
struct Span {
  const void* p;
  long long rows, cols, ld;
  int elem;
  bool out;
};

constexpr long long kMaxLd = 1LL << 28;  // keeps every byte offset of 2^31 rows below 2^62

// Every array in use is element-aligned device (or managed) memory of the current device, its
// stride in [0, kMaxLd]; rows of an output do not overlap one another, and no output shares
// memory with another argument (rows of two arrays may interleave, as column ranges of one wider
// array do). Inputs may have any stride, 0 (one row for all) included. Enqueues nothing; what
// needs no device is checked first.
int check_spans(const Span* s, int n);

// The status words of the waits inside the lookup's and the feed-forward block's kernels, read and
// cleared (waits for the stream).
cudaError_t lookup_status_take(unsigned int* out, cudaStream_t st);
cudaError_t ffn_status_take(unsigned int* out, cudaStream_t st);

}  // namespace rows
}  // namespace splat
