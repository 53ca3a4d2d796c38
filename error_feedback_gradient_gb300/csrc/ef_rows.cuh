// Shared internals of the training losses (ef_logits.cu, ef_distill.cu,
// ef_balance.cu): logits of three types, ordered keys, block reductions in a
// fixed order, and the host's argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "ef_common.cuh"

namespace ef {

// ---------------------------------------------------------------------------
// device side
// ---------------------------------------------------------------------------

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// 2^x by the special-function unit: relative error at most 2^-22, results
// below 2^-126 flushed to 0 (such terms are nothing against a sum of at least
// 1, and nothing in a gradient's type).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(a - b) for log-domain a, b; 0 where a is -Inf (b may be too).
__device__ __forceinline__ float exp_diff(float a, float b) {
  return a == kNegInf ? 0.0f : expf(a - b);
}

// Reference for 2^(x - m): the maximum itself, or 0 where nothing is left (so
// that masked entries give 2^-Inf = 0 and a NaN stays one).
__device__ __forceinline__ float finite_ref(float m) { return m == kNegInf ? 0.0f : m; }

// Order-preserving 32-bit key of a float: ascending with its value, every NaN
// above +Inf, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order_key(-Inf)

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Block maximum / sum, the same value in every thread; the sum's order is
// fixed by the block's size.  `scratch`: 32 floats.  Contain __syncthreads().
__device__ __forceinline__ float block_max(float v, float* scratch) {
  v = warp_max(v);
  if (lane_id() == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_max(lane_id() < (blockDim.x >> 5) ? scratch[lane_id()] : kNegInf);
  __syncthreads();
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* scratch) {
  v = warp_sum(v);
  if (lane_id() == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_sum(lane_id() < (blockDim.x >> 5) ? scratch[lane_id()] : 0.0f);
  __syncthreads();
  return v;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline int dtype_size(int32_t dtype) {
  return dtype == EF_DTYPE_F32 ? 4 : dtype == EF_DTYPE_BF16 || dtype == EF_DTYPE_F16 ? 2 : 0;
}

// Bytes between the first and one past the last element of a row buffer.
inline size_t rows_bytes(int64_t rows, int64_t cols, int64_t stride, int size) {
  return rows <= 0 || cols <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)stride + (size_t)cols) * size;
}
inline bool aligned_to(const void* p, int size) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1)) == 0;
}

// Sizes and scalars shared by the row-packet calls.
inline ef_status check_rows(int32_t dtype, int64_t rows, int64_t vocab, int64_t stride, int32_t k,
                            float tau) {
  if (dtype_size(dtype) == 0) return EF_ERR_ARG;
  if (rows < 0 || rows >= (1ll << 31) || vocab < 0 || vocab > (1ll << 30) || stride < vocab ||
      stride > (1ll << 40))
    return EF_ERR_SIZE;
  if (k < 0 || k > EF_MAX_ROW_PACKET || k > vocab) return EF_ERR_K;
  if (!std::isfinite(tau) || !(tau > 0.0f)) return EF_ERR_ARG;
  return EF_OK;
}

// A buffer of a call, for the pairwise overlap check.
struct Span {
  const void* p;
  size_t bytes;
  bool out;
};
inline bool any_overlap(const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((s[i].out || s[j].out) && overlaps(s[i].p, s[i].bytes, s[j].p, s[j].bytes)) return true;
  return false;
}

// `F` is called with a value of the element type.
template <typename F>
inline void with_dtype(int32_t dtype, F f) {
  if (dtype == EF_DTYPE_F32) f(float());
  else if (dtype == EF_DTYPE_BF16) f(__nv_bfloat16());
  else f(__half());
}

}  // namespace ef
