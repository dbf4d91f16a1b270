// lt_mv4.hpp -- products of a few vectors with a matrix of INT4 codes,
// y = x W^T (gfx950, wave64).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lt_types.hpp"

namespace lt {

struct Mv4Params {
  const uint8_t *w;          // packed codes, element e = r * cols + c
  const uint16_t *scales;
  const int8_t *zp;          // or NULL
  const uint16_t *x;
  void *y;
  uint64_t x_stride, y_stride;   // elements
  uint64_t group;
  uint32_t rows, cols, batch;
  uint32_t x_bf16, y_type;
};

// Any shape: one wave per row and block of 4 vectors, lane l taking columns
// l, l + 64, ..; sums per lane, then across the wave.
__global__ void __launch_bounds__(256) mv4_any_kernel(Mv4Params P) {
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t r = blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint32_t b0 = blockIdx.y * 4;
  if (r >= P.rows) return;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t c = lane; c < P.cols; c += 64) {
    const uint64_t e = (uint64_t)r * P.cols + c;
    const uint64_t g = e / P.group;
    const int q = (P.w[e >> 1] >> (4 * (e & 1))) & 15;
    const float w = (float)(q - (P.zp ? (int)P.zp[g] : 0)) * f32_of_f16(P.scales[g]);
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (b0 + k < P.batch) acc[k] = fmaf(w, f32_of_bits(P.x[(b0 + k) * P.x_stride + c], P.x_bf16), acc[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; k++) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) acc[k] += __shfl_xor(acc[k], d);
    if (lane == 0 && b0 + k < P.batch) store_as(P.y, (b0 + k) * P.y_stride + r, acc[k], P.y_type);
  }
}

}  // namespace lt
