// norm.hpp -- sums of the gradient norms and the clip coefficient, shared by
// the norm, clip and bucket all-reduce kernels.
//
// A norm is joined from parts: L2 adds squares, L1 adds magnitudes, the
// largest magnitude takes maxima. Sums are held in 64 bits from the first
// element on: the square of any fp32 value is exact there (48 of 53 bits) and
// neither overflows nor vanishes, so a norm is finite whenever its value fits
// fp32, tiny gradients keep theirs, and the order of the additions changes
// nothing that survives the final rounding to fp32 but in rare ties. These
// kernels wait for memory; the 64-bit additions cost no time.
#pragma once

#include "internal.hpp"

namespace ddpsim {

#if defined(__HIPCC__)

template <int NT>
struct NormSum;

template <>
struct NormSum<DDP_NORM_L2> {
  double v = 0.0;
  __device__ __forceinline__ void add(float x) {
    const double d = x;
    v = __builtin_fma(d, d, v);  // d * d is exact
  }
  __device__ __forceinline__ void join(const NormSum &o) { v = v + o.v; }
  __device__ __forceinline__ NormSum across(int mask) const {
    NormSum o;
    o.v = __shfl_xor(v, mask, 64);
    return o;
  }
  __device__ __forceinline__ double part() const { return v; }
  __device__ __forceinline__ void join_part(double d) { v = v + d; }
  __device__ __forceinline__ float norm() const { return static_cast<float>(sqrt(v)); }
};

template <>
struct NormSum<DDP_NORM_L1> {
  double v = 0.0;
  __device__ __forceinline__ void add(float x) { v = v + static_cast<double>(fabsf(x)); }
  __device__ __forceinline__ void join(const NormSum &o) { v = v + o.v; }
  __device__ __forceinline__ NormSum across(int mask) const {
    NormSum o;
    o.v = __shfl_xor(v, mask, 64);
    return o;
  }
  __device__ __forceinline__ double part() const { return v; }
  __device__ __forceinline__ void join_part(double d) { v = v + d; }
  __device__ __forceinline__ float norm() const { return static_cast<float>(v); }
};

// Magnitudes as integers: without the sign bit, the bits of fp32 values order
// like their magnitudes, infinity above every number and NaN above infinity,
// so the integer maximum keeps a NaN that a float maximum would drop.
template <>
struct NormSum<DDP_NORM_INF> {
  uint32_t v = 0;
  __device__ __forceinline__ void add(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    v = u > v ? u : v;
  }
  __device__ __forceinline__ void join(const NormSum &o) { v = o.v > v ? o.v : v; }
  __device__ __forceinline__ NormSum across(int mask) const {
    NormSum o;
    o.v = static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), mask, 64));
    return o;
  }
  __device__ __forceinline__ double part() const { return __uint_as_float(v); }
  __device__ __forceinline__ void join_part(double d) { add(static_cast<float>(d)); }
  __device__ __forceinline__ float norm() const { return __uint_as_float(v); }
};

// Every lane receives the whole wave's sum.
template <int NT>
__device__ __forceinline__ void join_wave(NormSum<NT> &s) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) s.join(s.across(m));
}

// min(1, max_norm / (norm + eps)) in fp32, one correctly rounded division.
// A norm of zero and an infinite bound leave the gradients; a NaN norm makes
// the coefficient NaN, an infinite one zero.
__device__ __forceinline__ float clip_coefficient(float norm, float max_norm, float eps) {
  if (norm == 0.0f || max_norm == __builtin_inff()) return 1.0f;
  const float c = max_norm / (norm + eps);
  return c >= 1.0f ? 1.0f : c;
}

#endif  // __HIPCC__

}  // namespace ddpsim
