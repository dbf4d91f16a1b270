// lt_mv4.hip -- liblt's entry point for products with INT4 matrices:
// argument checks and launches.  Nothing here allocates, synchronizes or
// keeps state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lt.h"
#include "lt_args.hpp"
#include "lt_mv4.hpp"

extern "C" {

lt_status lt_gemv_int4(const uint8_t *packed, const uint16_t *scales, const int8_t *zp, uint64_t rows,
                       uint64_t cols, uint64_t group, const void *x, uint64_t x_stride, uint32_t batch,
                       lt_dtype x_type, void *y, uint64_t y_stride, lt_dtype y_type, void *stream) {
  if (!packed || !scales || !x || !y || batch == 0 || x_stride < cols || y_stride < rows) return LT_ERR_INVALID_ARG;
  if (!lt::shape_ok(rows, cols, group) || (rows * cols) % 2 != 0) return LT_ERR_INVALID_ARG;
  if (x_type != LT_F16 && x_type != LT_BF16) return LT_ERR_INVALID_ARG;
  if (y_type != LT_F16 && y_type != LT_BF16 && y_type != LT_F32) return LT_ERR_INVALID_ARG;
  if (((uintptr_t)x & 1) != 0 || ((uintptr_t)scales & 1) != 0) return LT_ERR_INVALID_ARG;
  if (((uintptr_t)y & (y_type == LT_F32 ? 3 : 1)) != 0) return LT_ERR_INVALID_ARG;
  if (batch > 64 || rows > 0x7FFFFFFFull || cols > 0x7FFFFFFFull) return LT_ERR_UNSUPPORTED;
  lt::Mv4Params P;
  P.w = packed;
  P.scales = scales;
  P.zp = zp;
  P.x = (const uint16_t *)x;
  P.y = y;
  P.x_stride = x_stride;
  P.y_stride = y_stride;
  P.group = group;
  P.rows = (uint32_t)rows;
  P.cols = (uint32_t)cols;
  P.batch = batch;
  P.x_bf16 = x_type == LT_BF16;
  P.y_type = y_type;
  hipLaunchKernelGGL(lt::mv4_any_kernel, dim3((P.rows + 3) / 4, (batch + 3) / 4), dim3(256), 0, (hipStream_t)stream,
                     P);
  return hipGetLastError() == hipSuccess ? LT_OK : LT_ERR_LAUNCH;
}

}  // extern "C"
