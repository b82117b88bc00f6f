// Activations of the training operators and 16-byte accesses to float32 / bf16 / f16 rows.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/qha.h"

namespace qha {

// exp(-z) and 1 / x on the transcendental units.  The exponent z log2(e) is rounded once, so exp(-z) is off by
// 1.5 |z| u of itself (u = 2^-24); where it matters it is multiplied by a sigmoid's slope, which
// falls faster than |z| grows, and sigmoids stay within 2 u.  Past exp's range the sigmoid is 0.
__device__ __forceinline__ float exp_neg(float z) { return __builtin_amdgcn_exp2f(fminf(z * -1.44269504088896341f, 127.0f)); }
__device__ __forceinline__ float sigmoid(float z) { return z == z ? __builtin_amdgcn_rcpf(1.0f + exp_neg(z)) : z; }

// act(z); `act` is uniform over a launch, so the branch costs one scalar test.  ReLU asks for z <= 0, which NaN is
// not: it stays NaN, with slope 1.
__device__ __forceinline__ float activate(float z, int32_t act) {
  if (act == QHA_ACT_RELU) return z <= 0.0f ? 0.0f : z;
  if (act == QHA_ACT_SILU) return z * sigmoid(z);
  if (act == QHA_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  return z;
}

// act(z) and act'(z).
__device__ __forceinline__ float activate_both(float z, int32_t act, float* slope) {
  if (act == QHA_ACT_RELU) {
    *slope = z <= 0.0f ? 0.0f : 1.0f;
    return z <= 0.0f ? 0.0f : z;
  }
  if (act == QHA_ACT_SILU) {
    const float s = sigmoid(z);
    *slope = s * (1.0f + z * (1.0f - s));
    return z * s;
  }
  if (act == QHA_ACT_GELU) {
    const float cdf = 0.5f * (1.0f + erff(z * 0.70710678118654752f));
    *slope = cdf + z * (0.39894228040143268f * exp_neg(0.5f * z * z));
    return z * cdf;
  }
  *slope = 1.0f;
  return z;
}

// dz = dy act'(z), z = w xhat + b; for ReLU the sign of z is that of the float64 value.
__device__ __forceinline__ float grad_z(float dy, float x, float mean, float rstd, float xhat, float w, float b,
                                        int32_t act) {
  if (act == QHA_ACT_NONE) return dy;
  if (act == QHA_ACT_RELU) {
    const double z = (static_cast<double>(x) - static_cast<double>(mean)) * static_cast<double>(rstd) *
                         static_cast<double>(w) + static_cast<double>(b);
    return z <= 0.0 ? 0.0f : dy;
  }
  float slope;
  activate_both(xhat * w + b, act, &slope);
  return dy * slope;
}

// 16 bytes of T: N elements, converted to and from float32 (one rounding, to nearest even).  Results leave as
// streaming stores, which keep the inputs still to be read in the caches (rows of 300k x 128 float32 54 against 62 us).
template <typename T>
struct Pack {
  static constexpr int N = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(N)));
  typedef float wide __attribute__((ext_vector_type(N)));
  static __device__ __forceinline__ wide load(const T* p) {
    return __builtin_convertvector(*reinterpret_cast<const vec*>(p), wide);
  }
  static __device__ __forceinline__ void store(T* p, wide x) {
    __builtin_nontemporal_store(__builtin_convertvector(x, vec), reinterpret_cast<vec*>(p));
  }
};

}  // namespace qha
