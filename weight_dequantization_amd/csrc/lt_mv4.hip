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
  hipLaunchKernelGGL(kernel, dim3((P.rows + 16 * RT - 1) / (16 * RT)), dim3(64 * NW), lds, s, P);
  return true;
}

// The workgroup's shape by the number of vectors.  Two tiles of rows a
// workgroup halve what x costs (40 us against 51 at 8192 x 28672, 16
// vectors); with fewer rows than fill the CUs that way, one.  Blocks of 256
// columns give whole 128-byte lines of W (34 us against 40, 8 vectors); with
// small groups the registers of their scales would halve the waves (13.7 us
// against 15.3 at 4999 x 8160, groups of 32, 13 vectors), and so would more
// than 16 vectors.
template <bool BF16, int GS, bool ZP>
bool launch_shape(const lt::Mv4Params &P, hipStream_t s) {
  constexpr int S = GS == 4 ? 256 : 128;
  if (P.batch > 32) return launch_tiles<BF16, 4, 2, GS, ZP, 4, 64, 128>(P, s);
  if (P.batch > 16) return launch_tiles<BF16, 2, 2, GS, ZP, 8, 32, 128>(P, s);
  if (P.rows > 4096) {
    if (P.batch > 8) return launch_tiles<BF16, 1, 2, GS, ZP, 8, 16, S>(P, s);
    if (P.batch > 4) return launch_tiles<BF16, 1, 2, GS, ZP, 8, 8, S>(P, s);
    return launch_tiles<BF16, 1, 2, GS, ZP, 8, 4, S>(P, s);
  }
  if (P.batch > 8) return launch_tiles<BF16, 1, 1, GS, ZP, 8, 16, S>(P, s);
  return launch_tiles<BF16, 1, 1, GS, ZP, 8, 8, S>(P, s);
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
