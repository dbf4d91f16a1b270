// lt_types.hpp -- 16-bit element types on the device: fp16 and bf16 bits to
// fp32 (exact) and back (round to nearest even); the order of a wave's LDS
// accesses.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lt.h"

namespace lt {

__device__ __forceinline__ float f32_of_f16(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
__device__ __forceinline__ float f32_of_bf16(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
__device__ __forceinline__ float f32_of_bits(uint16_t v, bool bf16) { return bf16 ? f32_of_bf16(v) : f32_of_f16(v); }

__device__ __forceinline__ uint16_t f16_of_f32(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ __forceinline__ uint16_t bf16_of_f32(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t bits_of_f32(float v, bool bf16) { return bf16 ? bf16_of_f32(v) : f16_of_f32(v); }

// element i of an array of lt_dtype `type`
__device__ __forceinline__ void store_as(void *p, uint64_t i, float v, uint32_t type) {
  if (type == LT_F32) {
    ((float *)p)[i] = v;
  } else {
    ((uint16_t *)p)[i] = bits_of_f32(v, type == LT_BF16);
  }
}

// Orders this wave's LDS accesses by different lanes (the hardware keeps the
// order of one wave's operations; this keeps the compiler's).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace lt
