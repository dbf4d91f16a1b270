// lt_mv4.hip -- liblt's entry point for products with INT4 matrices:
// argument checks and launches.  Nothing here allocates, synchronizes or
// keeps state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lt.h"
#include "lt_args.hpp"
#include "lt_mv4.hpp"

namespace {

template <bool BF16, bool ZP>
void launch_one(const lt::Mv4Params &P, hipStream_t s) {
  // The waves of a workgroup lie side by side over the columns.  x costs as
  // much to load as 4 rows (2 of codes, 2 of what else a row takes), so a
  // wave takes several 4-row steps as soon as the grid still gives every CU
  // about 24 waves: at 8192 x 28672 4 steps take 26.7 us, 2 take 34.4; at
  // 1024 x 8192 1 step takes 3.4 us, 2 take 4.0.
  const uint32_t blocks = (P.cols + 2047) / 2048, rounds = (blocks + 15) / 16;
  const uint32_t parts = (blocks + rounds - 1) / rounds, downs = parts >= 4 ? 1 : 4 / parts;
  const uint64_t waves = (uint64_t)((P.rows + 3) / 4) * parts;
  uint64_t steps = waves / 6144;
  steps = steps < 1 ? 1 : steps > 16 ? 16 : steps;
  const uint32_t per = (uint32_t)(4 * steps * downs);
  hipLaunchKernelGGL((lt::mv4_one_kernel<BF16, ZP>), dim3((P.rows + per - 1) / per), dim3(64 * parts * downs),
                     parts * per * 4, s, P, per, parts);
}

template <bool BF16, int MT, int RT, int GS, bool ZP, int NW, int XR, int S>
bool launch_tiles(const lt::Mv4Params &P, hipStream_t s) {
  constexpr uint32_t own = NW * lt::mv4_wave_lds<RT, XR, S>, join = NW * RT * MT * 1024;
  constexpr uint32_t lds = own > join ? own : join;
  auto kernel = lt::mv4_kernel<BF16, MT, RT, GS, ZP, NW, XR, S>;
  if (lds > 65536 &&
      hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
    return false;
  const uint32_t blocks = ((P.rows + 16 * RT - 1) / (16 * RT) + 7) / 8 * 8 * ((P.batch + XR - 1) / XR);
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(64 * NW), lds, s, P);
  return true;
}

// The workgroup's shape.  Two tiles of rows a workgroup halve what x costs
// and two tiles of vectors what W's operands cost, as long as every CU still
// gets a workgroup (40.7 us against 49.7 with one tile of rows at 8192 x
// 28672, 16 vectors, but 10.2 against 8.7 at 4096 x 8192; 15.6 us against
// 18.6 with two blocks of 16 vectors at 8192 x 8192, 32 vectors, but 7.5
// against 6.4 at 4096 x 4096).  16 waves with blocks of 128 columns hide
// more of each other's waits than 8 with 256 (11.5 us against 12.8 at 8192 x
// 8192, 16 vectors; 8.7 against 9.7 at 4096 x 8192), but long rows in many
// workgroups want whole 128-byte lines of W (40.7 us against 47.3 at 8192 x
// 28672; 27.2 against 30.3 at 5000 x 28672).
template <bool BF16, int GS, bool ZP>
bool launch_shape(const lt::Mv4Params &P, hipStream_t s) {
  const bool lines = P.cols > 16384;
  if (P.batch > 16 && (uint64_t)P.rows * ((P.batch + 31) / 32) > 4096)
    return launch_tiles<BF16, 2, 2, GS, ZP, 8, 32, 128>(P, s);
  if ((uint64_t)P.rows * ((P.batch + 15) / 16) <= 4096)
    return P.batch > 8 ? launch_tiles<BF16, 1, 1, GS, ZP, 16, 16, 128>(P, s)
                       : launch_tiles<BF16, 1, 1, GS, ZP, 16, 8, 128>(P, s);
  if (P.batch > 8)
    return lines ? launch_tiles<BF16, 1, 2, GS, ZP, 8, 16, 256>(P, s) : launch_tiles<BF16, 1, 2, GS, ZP, 16, 16, 128>(P, s);
  if (P.batch > 4)
    return lines ? launch_tiles<BF16, 1, 2, GS, ZP, 8, 8, 256>(P, s) : launch_tiles<BF16, 1, 2, GS, ZP, 16, 8, 128>(P, s);
  return lines ? launch_tiles<BF16, 1, 2, GS, ZP, 8, 4, 256>(P, s) : launch_tiles<BF16, 1, 2, GS, ZP, 16, 4, 128>(P, s);
}

template <bool BF16, bool ZP>
bool launch_fast(const lt::Mv4Params &P, hipStream_t s) {
  if (P.batch == 1) {
    launch_one<BF16, ZP>(P, s);
    return true;
  }
  const uint64_t gc = P.group < P.cols ? P.group : P.cols;
  if (gc % 128 == 0 || gc == P.cols) return launch_shape<BF16, 4, ZP>(P, s);
  return gc % 64 == 0 ? launch_shape<BF16, 2, ZP>(P, s) : launch_shape<BF16, 1, ZP>(P, s);
}

}  // namespace

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
  P.group_shift = lt::shift_of(group);
  P.rows = (uint32_t)rows;
  P.cols = (uint32_t)cols;
  P.batch = batch;
  P.x_bf16 = x_type == LT_BF16;
  P.y_type = y_type;
  hipStream_t s = (hipStream_t)stream;
  const uint64_t gc = group < cols ? group : cols;
  // 32 neighbouring columns make one 16-byte load of codes, and share a group
  const bool fast = cols % 32 == 0 && gc % 32 == 0 && lt::aligned16(packed) && lt::aligned16(x) &&
                    (batch == 1 || x_stride % 8 == 0);
  if (fast) {
    const bool ok = P.x_bf16 ? (zp ? launch_fast<true, true>(P, s) : launch_fast<true, false>(P, s))
                             : (zp ? launch_fast<false, true>(P, s) : launch_fast<false, false>(P, s));
    if (!ok) return LT_ERR_LAUNCH;
  } else {
    hipLaunchKernelGGL(lt::mv4_any_kernel, dim3((P.rows + 3) / 4, (batch + 3) / 4), dim3(256), 0, s, P);
  }
  return hipGetLastError() == hipSuccess ? LT_OK : LT_ERR_LAUNCH;
}

}  // extern "C"
