// What the tiled matrix products share: vector types, the matrix instructions, and loads from memory into LDS.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace qha {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kXcds = 8;        // accelerator complex dies, each with its own L2

template <typename T>
__device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mma<__bf16>(s16x8 a, s16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mma<_Float16>(s16x8 a, s16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ f32x4 mma16(s16x8 a, s16x8 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mma16<__bf16>(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma16<_Float16>(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Waits for this wavefront's loads into LDS; a barrier after it makes them visible to the block.
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Waits until at most N of them (of the last ones) are on their way.
template <int N>
__device__ __forceinline__ void loads_left() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }

// 16 bytes a lane from memory to LDS, lane i of the wavefront to `to` + 16 i.  Written as assembly because
// the compiler would wait for all such loads before any LDS read that it cannot tell apart from their
// destination (the transposing reads), and so undo the double buffering; nothing comes back in a
// vector register, and loads_done() waits.  m0, which holds the destination, is an output, so that the compiler
// knows it to have changed (it takes no reserved register in a list of clobbers).
__device__ __forceinline__ void load_to_lds(const uint16_t* from, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : "={m0}"(m0) : "v"(from), "s"(to) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const uint16_t* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint16_t*)p));
}

}  // namespace
}  // namespace qha
