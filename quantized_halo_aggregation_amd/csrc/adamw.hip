// AdamW over many tensors in one launch, with moments in float32 or in 8-bit block codes.
//
// Mathematics: m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2, p = p (1 - lr wd) - lr m^ / (sqrt(v^) + eps)
// with m^ = m / (1 - b1^t), v^ = v / (1 - b2^t).  8-bit moments are companded per block of 256 elements:
// m = s sign(c) (c / 127)^2 and v = s (c / 255)^4, which spaces the codes by about 2 / c of the value, so
// a small moment beside a large one keeps a code; s is the block's largest magnitude.
//
// Bound: memory.  Per element 28 bytes move with float32 moments and gradients, 16 with 8-bit
// moments, 16-bit gradients and a 16-bit copy.  The 8-bit form's arithmetic is float64, so that a code is the same
// whichever way its inputs were summed; most of it hides behind memory, not all: it reaches 4.7 TB/s.
//
// 302M elements with float32 moments and gradients: 1.46 to 1.60 ms by card (5.3 to 5.8 TB/s; a large copy reaches 5.0).  201M with
// 8-bit moments, bf16 gradients and copies: 0.69 ms (4.7 TB/s), and 0.35 ms to read the moments back (5.8 TB/s).
//
// Mapping: a block of 256 threads takes chunks of 1024 consecutive elements, four per thread (16-byte
// accesses), so that one wavefront holds exactly one 256-element code block and finds its largest
// magnitude with wavefront reductions.  The tensors' pointers travel in the kernel arguments (48
// tensors in one launch, nothing copied to the device), and a block finds its tensor by comparing their
// first blocks in one step.
#include "qha_internal.hpp"

#include "../../include/qha.h"

#pragma clang fp contract(off)

namespace qha {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef int8_t i8x4 __attribute__((ext_vector_type(4)));
typedef uint8_t u8x4 __attribute__((ext_vector_type(4)));

// Four consecutive elements from index i on of an array of n, as one access when `vec` (the array is
// aligned and the four are inside), else element by element (0 past the end).
template <typename V, typename E>
__device__ __forceinline__ V load4(const void* p, int64_t i, int64_t n, bool vec) {
  const E* q = static_cast<const E*>(p) + i;
  if (vec) return *reinterpret_cast<const V*>(q);
  V r = {};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) r[j] = q[j];
  return r;
}

template <typename V, typename E>
__device__ __forceinline__ void store4(void* p, int64_t i, int64_t n, bool vec, V x) {
  E* q = static_cast<E*>(p) + i;
  if (vec) {
    *reinterpret_cast<V*>(q) = x;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) q[j] = x[j];
}

__device__ __forceinline__ f32x4 load_grad(const void* g, int32_t type, int64_t i, int64_t n, bool vec) {
  if (type == QHA_F32) return load4<f32x4, float>(g, i, n, vec);
  if (type == QHA_BF16) return __builtin_convertvector((load4<bf16x4, __bf16>(g, i, n, vec)), f32x4);
  return __builtin_convertvector((load4<f16x4, _Float16>(g, i, n, vec)), f32x4);
}

__device__ __forceinline__ void store_copy(void* c, int32_t type, int64_t i, int64_t n, bool vec, f32x4 p) {
  if (type == QHA_BF16) store4<bf16x4, __bf16>(c, i, n, vec, __builtin_convertvector(p, bf16x4));
  else if (type == QHA_F16) store4<f16x4, _Float16>(c, i, n, vec, __builtin_convertvector(p, f16x4));
  else store4<f32x4, float>(c, i, n, vec, p);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_across(uint32_t x) {
  const uint32_t y = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(x), static_cast<int>(x), CTRL, ROWS, 0xf, false));
  return x > y ? x : y;
}

// The wavefront's largest x, by exchanges within rows of 16 lanes and broadcasts between them.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max_across<0xB1, 0xf>(x);         // lane ^ 1
  x = max_across<0x4E, 0xf>(x);         // lane ^ 2
  x = max_across<0x141, 0xf>(x);        // mirrored in 8
  x = max_across<0x140, 0xf>(x);        // mirrored in 16
  x = max_across<0x142, 0xa>(x);        // rows 1 and 3 take the row before
  x = max_across<0x143, 0xc>(x);        // the upper half takes lane 31
  return __builtin_amdgcn_readlane(x, 63);
}

__device__ __forceinline__ double lane_double(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// The largest of the wavefront's four-element shares of |x|, whose float32 roundings are m: as float32
// (*rounded), and as the float64 value.  Float32 magnitudes order as their bits do, with infinities
// and NaN on top (*rounded then is not finite and the result unused); the lanes whose largest rounds to
// the wavefront's, almost always one, hold the float64 value.
__device__ __forceinline__ double wave_largest(const double (&x)[4], f32x4 m, float* rounded) {
  uint32_t own = 0;
  double wide = 0.0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = __float_as_uint(m[j]) & 0x7FFFFFFFu;
    own = own > b ? own : b;
    wide = fmax(wide, fabs(x[j]));
  }
  const uint32_t top = wave_max(own);
  *rounded = __uint_as_float(top);
  const uint64_t who = __ballot(own == top);
  if ((who & (who - 1)) == 0 || top == 0) return lane_double(wide, __builtin_ctzll(who));
  wide = own == top ? wide : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) wide = fmax(wide, __shfl_xor(wide, o, 64));
  return wide;
}

// Nearest codes of |x| inv (inv = 1 / largest): TOP (|x| inv)^(1/POWER), rounded.  The root is taken in
// float32 (off by less than 7e-5 codes); where any of the four is within 1e-4 of a half-way point all are
// decided in float64 on the ratios, whose half-way points are ((c + 1/2) / TOP)^POWER.  16-bit gradients put
// ratios exactly on some of those (1/4 is code 63 1/2 of 127), where the last bit of the ratio would
// decide: a ratio has to be over the point by 2^-40 of it to go up.
template <int TOP, int POWER>
__device__ __forceinline__ void nearest_codes(const double (&x)[4], double inv, int (&code)[4]) {
  float t[4];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float r = __builtin_amdgcn_sqrtf(static_cast<float>(fabs(x[j]) * inv));
    if (POWER == 4) r = __builtin_amdgcn_sqrtf(r);
    t[j] = r * TOP;
    const float up = rintf(t[j]);
    code[j] = static_cast<int>(up);
    near = near || fabsf(t[j] - up) > 0.4999f;
  }
  if (near) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double base = floor(static_cast<double>(t[j]));
      double e = (base + 0.5) * (1.0 / TOP);
      e *= e;
      if (POWER == 4) e *= e;
      // away from a half-way point this is the rounding above
      const bool up = fabs(x[j]) * inv > e * (1.0 + 0x1p-40);
      code[j] = min(static_cast<int>(base) + (up ? 1 : 0), TOP);
    }
  }
}

__device__ __forceinline__ f32x4 new_params(const AdamArgs& a, f32x4 p, f32x4 m, f32x4 v) {
  f32x4 r;
  // the reciprocal is the transcendental unit's, off by at most one step
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r[j] = p[j] * a.decay - a.step_size * (m[j] * __builtin_amdgcn_rcpf(sqrtf(v[j]) * a.root_c2 + a.eps));
  return r;
}

template <int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(AdamArgs a) {
  // the tensor whose chunks include this block: the last one that starts at or before it (at most 48
  // tensors, compared by one lane each: the kernel's arguments are read over a slow path, so in one go)
  const int ln = threadIdx.x & 63;
  const uint32_t start = ln < a.n_tensors ? a.first[ln] : 0xFFFFFFFFu;
  const int lo = __builtin_amdgcn_readfirstlane(__popcll(__ballot(start <= blockIdx.x)) - 1);
  const AdamTensor t = a.t[lo];
  const uintptr_t wide = reinterpret_cast<uintptr_t>(t.p) | (BITS == 32 ? reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v) : 0) |
                         (a.grad_type == QHA_F32 ? reinterpret_cast<uintptr_t>(t.g) : 0) | (a.copy_type == QHA_F32 ? reinterpret_cast<uintptr_t>(t.copy) : 0);
  const uintptr_t half = (a.grad_type == QHA_F32 ? 0 : reinterpret_cast<uintptr_t>(t.g)) | (a.copy_type == QHA_F32 ? 0 : reinterpret_cast<uintptr_t>(t.copy));
  const uintptr_t quarter = BITS == 8 ? reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v) : 0;
  const bool aligned = (wide & 15) == 0 && (half & 7) == 0 && (quarter & 3) == 0;
  const int64_t begin = static_cast<int64_t>(blockIdx.x - a.first[lo]) * a.passes * 1024;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int64_t i = begin + pass * 1024 + threadIdx.x * 4;
    // a wavefront's 256 elements are one code block, so this leaves whole wavefronts only
    if (begin + pass * 1024 + (threadIdx.x & ~63u) * 4 >= t.n) return;
    const bool vec = aligned && i + 4 <= t.n;
    f32x4 p = load4<f32x4, float>(t.p, i, t.n, vec);
    f32x4 g = load_grad(t.g, a.grad_type, i, t.n, vec);
    g *= a.grad_scale;
    f32x4 m, v;
    if (BITS == 32) {
      const float b1 = static_cast<float>(a.beta1), b2 = static_cast<float>(a.beta2);
      const float o1 = static_cast<float>(1.0 - a.beta1), o2 = static_cast<float>(1.0 - a.beta2);
      m = load4<f32x4, float>(t.m, i, t.n, vec);
      v = load4<f32x4, float>(t.v, i, t.n, vec);
      m = m * b1 + g * o1;
      v = v * b2 + (g * g) * o2;
      store4<f32x4, float>(t.m, i, t.n, vec, m);
      store4<f32x4, float>(t.v, i, t.n, vec, v);
    } else {
      const int64_t blk = i / kAdamBlock;
      const i8x4 cm = load4<i8x4, int8_t>(t.m, i, t.n, vec);
      const u8x4 cv = load4<u8x4, uint8_t>(t.v, i, t.n, vec);
      const double sm = static_cast<double>(t.ms[blk]);
      const double sv = static_cast<double>(t.vs[blk]);
      double xm[4], xv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = cm[j];
        const uint32_t u = static_cast<uint32_t>(cv[j]) * cv[j];
        const double gd = static_cast<double>(g[j]);
        // every product and sum rounded as the formula is written, so that a float64 program gets these very
        // moments: 0.9 a + 0.1 b lies half-way between two float32 scales often enough for the last bit to matter
        const double old_m = sm * static_cast<double>(c * (c < 0 ? -c : c)) * (1.0 / (127.0 * 127.0));
        const double old_v = sv * static_cast<double>(u * u) * (1.0 / (255.0 * 255.0 * 255.0 * 255.0));
        xm[j] = a.beta1 * old_m + (1.0 - a.beta1) * gd;
        xv[j] = a.beta2 * old_v + (1.0 - a.beta2) * (gd * gd);
        m[j] = static_cast<float>(xm[j]);
        v[j] = static_cast<float>(xv[j]);
      }
      float sm32, sv32;
      i8x4 nm = {};
      u8x4 nv = {};
      int code[4];
      const double top_m = wave_largest(xm, m, &sm32);
      if (__builtin_isfinite(sm32)) {
        nearest_codes<127, 2>(xm, sm32 > 0.0f ? 1.0 / top_m : 0.0, code);
#pragma unroll
        for (int j = 0; j < 4; ++j) nm[j] = static_cast<int8_t>(xm[j] < 0.0 ? -code[j] : code[j]);
      } else {
        sm32 = __builtin_nanf("");
      }
      const double top_v = wave_largest(xv, v, &sv32);
      if (__builtin_isfinite(sv32)) {
        nearest_codes<255, 4>(xv, sv32 > 0.0f ? 1.0 / top_v : 0.0, code);
#pragma unroll
        for (int j = 0; j < 4; ++j) nv[j] = static_cast<uint8_t>(xv[j] > 0.0 ? max(code[j], 1) : 0);
      } else {
        sv32 = __builtin_nanf("");
      }
      store4<i8x4, int8_t>(t.m, i, t.n, vec, nm);
      store4<u8x4, uint8_t>(t.v, i, t.n, vec, nv);
      if ((threadIdx.x & 63) == 0) {
        t.ms[blk] = sm32;
        t.vs[blk] = sv32;
      }
    }
    p = new_params(a, p, m, v);
    store4<f32x4, float>(t.p, i, t.n, vec, p);
    if (t.copy) store_copy(t.copy, a.copy_type, i, t.n, vec, p);
  }
}

__global__ __launch_bounds__(256) void adamw_values_kernel(const int8_t* m, const float* ms, float* m_out,
                                                           const uint8_t* v, const float* vs, float* v_out,
                                                           int64_t n) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const uintptr_t al = reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(v);
  const uintptr_t ao = reinterpret_cast<uintptr_t>(m_out) | reinterpret_cast<uintptr_t>(v_out);
  const bool vec = i + 4 <= n && (al & 3) == 0 && (ao & 15) == 0;
  const int64_t blk = i / kAdamBlock;
  if (m) {
    const i8x4 c = load4<i8x4, int8_t>(m, i, n, vec);
    const double s = static_cast<double>(ms[blk]) * (1.0 / (127.0 * 127.0));
    f32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = static_cast<float>(s * static_cast<double>(c[j] * (c[j] < 0 ? -c[j] : c[j])));
    store4<f32x4, float>(m_out, i, n, vec, r);
  }
  if (v) {
    const u8x4 c = load4<u8x4, uint8_t>(v, i, n, vec);
    const double s = static_cast<double>(vs[blk]) * (1.0 / (255.0 * 255.0 * 255.0 * 255.0));
    f32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = static_cast<uint32_t>(c[j]) * c[j];
      r[j] = static_cast<float>(s * static_cast<double>(u * u));
    }
    store4<f32x4, float>(v_out, i, n, vec, r);
  }
}

}  // namespace

// 1024-element passes per block: one while the whole step has few enough of them that every block
// runs at once, else four, which quarters the look-ups of a block's tensor.
int32_t adamw_passes(int64_t elements) { return elements <= (8LL << 20) ? 1 : 4; }

hipError_t launch_adamw(const AdamArgs& a, int32_t state_bits, hipStream_t s) {
  const uint32_t blocks = a.first[a.n_tensors];
  if (blocks == 0) return hipSuccess;
  if (state_bits == 8) adamw_kernel<8><<<blocks, 256, 0, s>>>(a);
  else adamw_kernel<32><<<blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_adamw_values(const int8_t* m, const float* ms, float* m_out, const uint8_t* v, const float* vs,
                               float* v_out, int64_t n, hipStream_t s) {
  adamw_values_kernel<<<static_cast<uint32_t>((n + 1023) / 1024), 256, 0, s>>>(m, ms, m_out, v, vs, v_out, n);
  return hipGetLastError();
}

}  // namespace qha
