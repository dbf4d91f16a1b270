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
  uint32_t group_shift;          // log2(group) if a power of two, else 64
  uint32_t rows, cols, batch;
  uint32_t x_bf16, y_type;
};

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

// 8 codes of one dword as 4 pairs of x's type.  A nibble c in a byte is the
// fp8 (e4m3) value c * 2^-9, denormal below 8, so the scaled conversion with
// 2^9 gives c exactly, two a time: 7 operations for 8 codes, pairs (0,2)
// (4,6) (1,3) (5,7); mv4_vector puts the values of x in the same order.
template <bool BF16>
__device__ __forceinline__ uint4 mv4_codes(uint32_t w) {
  const uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;
  uint4 r;
  if constexpr (BF16) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, true));
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f, true));
  }
  return r;
}

__device__ __forceinline__ uint4 mv4_vector(uint4 v) {
  const uint32_t lo = 0x05040100u, hi = 0x07060302u;
  return make_uint4(__builtin_amdgcn_perm(v.y, v.x, lo), __builtin_amdgcn_perm(v.w, v.z, lo),
                    __builtin_amdgcn_perm(v.y, v.x, hi), __builtin_amdgcn_perm(v.w, v.z, hi));
}

typedef _Float16 hp2 __attribute__((ext_vector_type(2)));
typedef __bf16 bp2 __attribute__((ext_vector_type(2)));

template <bool BF16>
__device__ __forceinline__ float mv4_dot2(uint32_t a, uint32_t b, float c) {
  if constexpr (BF16)
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bp2, a), __builtin_bit_cast(bp2, b), c, false);
  else
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(hp2, a), __builtin_bit_cast(hp2, b), c, false);
}

// Sums over the 64 lanes of 4 values at once: swapping halves and rows of
// lanes folds the 4 registers into one whose 16-lane row k holds value
// (0, 2, 1, 3)[k], which 4 rotations within the rows then sum.
__device__ __forceinline__ float mv4_fold(float v0, float v1, float v2, float v3) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  auto bits = [](float f) { return __builtin_bit_cast(uint32_t, f); };
  auto sum = [](u2 s) {
    const uint32_t lo = s[0], hi = s[1];
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
  };
  const float a = sum(__builtin_amdgcn_permlane32_swap(bits(v0), bits(v1), false, false));
  const float b = sum(__builtin_amdgcn_permlane32_swap(bits(v2), bits(v3), false, false));
  float v = sum(__builtin_amdgcn_permlane16_swap(bits(a), bits(b), false, false));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xF, 0xF, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x124, 0xF, 0xF, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x122, 0xF, 0xF, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x121, 0xF, 0xF, true));
  return v;
}

// The form for one vector.  A wave keeps x of a block of 2048 columns in
// registers, lane l the 32 columns from 32 l, and goes down the rows of its
// workgroup: one 16-byte load a row (1 KiB side by side) whose 32 codes share
// a group.  The workgroup's parts * downs waves take the blocks and every
// downs-th 4 rows; rows' sums meet in LDS, [parts][per].  Bytes of W bound it:
// 8192 x 28672, groups of 128, 26.5 us, 4.6 TB/s of the 6.1 that a plain read
// reaches; 1024 x 1024 takes 3.6 us, the time of a launch.
template <bool BF16, bool ZP>
__global__ void __launch_bounds__(1024) mv4_one_kernel(Mv4Params P, uint32_t per, uint32_t parts) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  float *red = (float *)lds;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t part = wave % parts, down = wave / parts, downs = blockDim.x / 64 / parts;
  const uint32_t r0 = blockIdx.x * per, r1 = P.rows - r0 < per ? P.rows : r0 + per;
  const uint32_t gc = P.group < P.cols ? (uint32_t)P.group : P.cols;
  for (uint32_t first = part * 2048; first < P.cols; first += parts * 2048) {
    const uint32_t c = first + 32 * lane;
    const bool in = c < P.cols;
    const uint32_t cc = in ? c : 0;
    uint4 x[4];
    float xs = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      x[k] = in ? mv4_vector(((const uint4 *)(P.x + cc))[k]) : make_uint4(0, 0, 0, 0);
      if (ZP) {
        const uint32_t ones = BF16 ? 0x3F803F80u : 0x3C003C00u;
        xs = mv4_dot2<BF16>(x[k].x, ones, xs);
        xs = mv4_dot2<BF16>(x[k].y, ones, xs);
        xs = mv4_dot2<BF16>(x[k].z, ones, xs);
        xs = mv4_dot2<BF16>(x[k].w, ones, xs);
      }
    }
    const uint32_t gi = P.group_shift < 32 ? cc >> P.group_shift : cc / gc;
    for (uint32_t r = r0 + 4 * down; r < r1; r += 4 * downs) {
      uint4 d[4];
      float s[4], z[4], t[4];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const uint64_t row = r + k < P.rows ? r + k : P.rows - 1;
        const uint64_t e = row * P.cols, g0 = P.group_shift < 64 ? e >> P.group_shift : e / P.group;
        d[k] = *(const uint4 *)(P.w + e / 2 + cc / 2);
        s[k] = f32_of_f16(P.scales[g0 + gi]);
        z[k] = ZP ? (float)P.zp[g0 + gi] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const uint32_t w[4] = {d[k].x, d[k].y, d[k].z, d[k].w};
        t[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const uint4 q = mv4_codes<BF16>(w[i]);
          t[k] = mv4_dot2<BF16>(q.x, x[i].x, t[k]);
          t[k] = mv4_dot2<BF16>(q.y, x[i].y, t[k]);
          t[k] = mv4_dot2<BF16>(q.z, x[i].z, t[k]);
          t[k] = mv4_dot2<BF16>(q.w, x[i].w, t[k]);
        }
        t[k] = s[k] * (ZP ? fmaf(-z[k], xs, t[k]) : t[k]);
      }
      const float v = mv4_fold(t[0], t[1], t[2], t[3]);
      const uint32_t k = lane >> 4, at = r - r0 + ((k & 1) << 1 | k >> 1);
      if ((lane & 15u) == 0 && r0 + at < r1) {
        float *o = red + part * per + at;
        *o = first == part * 2048 ? v : *o + v;
      }
    }
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < r1 - r0; i += blockDim.x) {
    float v = 0.0f;
    for (uint32_t k = 0; k < parts; k++) v += red[k * per + i];
    store_as(P.y, r0 + i, v, P.y_type);
  }
}

template <bool BF16>
__device__ __forceinline__ f4 mv4_mfma(uint4 a, uint4 b, f4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// Four lanes 16 apart hold 4 dwords each: dword k of lane group g goes to
// dword g of lane group k.
__device__ __forceinline__ void mv4_transpose(uint32_t d[4]) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const u2 s = __builtin_amdgcn_permlane32_swap(d[i], d[i + 2], false, false);
    d[i] = s[0];
    d[i + 2] = s[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const u2 s = __builtin_amdgcn_permlane16_swap(d[i], d[i + 1], false, false);
    d[i] = s[0];
    d[i + 1] = s[1];
  }
}

// The matrix-core form.  The workgroup's NW waves share RT tiles of 16 rows of
// W and take blocks of S columns in turn.  A wave loads its block of W and
// of x with neighbouring lanes side by side in memory and turns both in its
// own part of LDS to operand order: lane (n, g) = (lane % 16, lane / 16) holds
// 32 codes of row n, columns 32 g .. + 31 of each half block, and vector n's
// values of the same columns.  16-byte pieces are stored at their index xor
// the row, so that neither side meets bank conflicts.  A product 16 x 16 x 32
// takes 16 vectors (A) and 16 rows (B), and leaves the sums of row n in lanes
// n, n + 16, .. (vectors 4 g .. 4 g + 3), where the lane has its own row's
// scale: y += s (sum q x - zp sum x), sum x out of one more product with a
// matrix of ones.  GS products share a group: 4 (groups of whole half blocks,
// or of whole rows), or 2 or 1 (groups of 64 or 32), for which dwords are
// first exchanged between lanes so that product k covers columns 32 k .. + 31.
// The waves add their sums through LDS in wave order.  What x costs bounds it
// (a workgroup loads all of x for its 32 rows, as much as W from 8 vectors on)
// and each wave's chain of load, LDS and product: 8192 x 28672 with 4, 8 and
// 16 vectors takes 28, 32 and 40 us, 32 vectors 57, 64 vectors 97; 4999 x 8160
// in groups of 32 with 13 vectors 13.4.  A second block in registers made each
// of them slower (16 vectors: 40.5), and so did buffer loads (40.2).
template <int RT, int XR, int S>
constexpr uint32_t mv4_wave_lds = RT * 8 * S + XR * 2 * S;

template <bool BF16, int MT, int RT, int GS, bool ZP, int NW, int XR, int S>
__global__ void __launch_bounds__(64 * NW) mv4_kernel(Mv4Params P) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int HB = S / 128;                // products' steps in a block
  constexpr int GPI = HB * (4 / GS);         // groups of a block in a row
  constexpr int CW = S / 32, CX = S / 8;     // 16-byte pieces of a row of W and of x
  constexpr int WI = RT * 16 * CW / 64, XI = (XR * CX + 63) / 64;   // load instructions
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, n = lane & 15u, g = lane >> 4;
  uint8_t *wl = lds + wave * mv4_wave_lds<RT, XR, S>, *xl = wl + RT * 8 * S;
  const uint32_t nblk = (P.cols + S - 1) / S;
  const uint32_t gc = P.group < P.cols ? (uint32_t)P.group : P.cols;   // columns of a row that share a scale
  const bool run = GPI == 1 || gc == 32 * GS;                          // a block's groups follow one another
  // blocks of rows in turn over the 8 L2s; the blocks of vectors of the same rows follow on the same one
  const uint32_t vblocks = (P.batch + XR - 1) / XR;
  const uint32_t pass = blockIdx.x / (8 * vblocks), in_pass = blockIdx.x % (8 * vblocks);
  const uint32_t r0 = (pass * 8 + in_pass % 8) * (RT * 16), v0 = in_pass / 8 * XR;
  if (r0 >= P.rows) return;
  const uint8_t *wp[WI];                     // rows of this lane's loads
#pragma unroll
  for (int i = 0; i < WI; i++) {
    const uint64_t r = r0 + i * (64 / CW) + lane / CW;
    wp[i] = P.w + (r < P.rows ? r : P.rows - 1) * P.cols / 2 + 16 * (lane % CW);
  }
  // lane l < 16 RT fetches the scales of row l
  const uint64_t sr = r0 + lane % (RT * 16) < P.rows ? r0 + lane % (RT * 16) : P.rows - 1;
  const uint64_t se = sr * P.cols, sg = P.group_shift < 64 ? se >> P.group_shift : se / P.group;
  const uint16_t *sp = P.scales + sg;
  const int8_t *zp = ZP ? P.zp + sg : nullptr;
  const uint16_t *xp[XI];
  bool xon[XI];
#pragma unroll
  for (int i = 0; i < XI; i++) {
    const uint32_t b = i * (64 / CX) + lane / CX;
    xon[i] = v0 + b < P.batch && b < XR;
    xp[i] = P.x + (xon[i] ? v0 + b : 0) * P.x_stride + 8 * (lane % CX);
  }
  auto turn = [](uint32_t r) { return CW == 8 ? r & 7u : (r >> 2) & 3u; };
  const f4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t one2 = BF16 ? 0x3F803F80u : 0x3C003C00u;
  const uint4 ones = make_uint4(one2, one2, one2, one2);
  f4 y[RT][MT];
#pragma unroll
  for (int rt = 0; rt < RT; rt++)
#pragma unroll
    for (int mt = 0; mt < MT; mt++) y[rt][mt] = zero;

  uint4 wd[WI], xd[XI];
  uint32_t sd[(GPI + 1) / 2], zd[(GPI + 3) / 4];
  auto fetch = [&](uint32_t blk) {
    const uint32_t c0 = blk * S;
    const bool win = c0 + 32 * (lane % CW) < P.cols, xin = c0 + 8 * (lane % CX) < P.cols;
#pragma unroll
    for (int i = 0; i < WI; i++) wd[i] = win ? *(const uint4 *)(wp[i] + c0 / 2) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < XI; i++) {
      xd[i] = make_uint4(0, 0, 0, 0);
      if (xon[i] && xin) xd[i] = *(const uint4 *)(xp[i] + c0);
    }
    if (lane < RT * 16) {
      if (run && c0 + S <= P.cols) {
        const uint32_t gi = P.group_shift < 32 ? c0 >> P.group_shift : c0 / gc;
        __builtin_memcpy(sd, sp + gi, 2 * GPI);
        if (ZP) __builtin_memcpy(zd, zp + gi, GPI);
      } else {
#pragma unroll
        for (int k = 0; k < (GPI + 1) / 2; k++) sd[k] = 0;
#pragma unroll
        for (int k = 0; k < (GPI + 3) / 4; k++) zd[k] = 0;
#pragma unroll
        for (int k = 0; k < GPI; k++) {
          const uint32_t c = c0 + k * (32 * GS);
          if (c < P.cols) {
            const uint32_t gi = P.group_shift < 32 ? c >> P.group_shift : c / gc;
            sd[k / 2] |= (uint32_t)sp[gi] << (16 * (k & 1));
            if (ZP) zd[k / 4] |= (uint32_t)(uint8_t)zp[gi] << (8 * (k & 3));
          }
        }
      }
    }
  };
  if (wave < nblk) fetch(wave);
  for (uint32_t blk = wave; blk < nblk; blk += NW) {
    wave_order();   // after the last block's reads
#pragma unroll
    for (int i = 0; i < WI; i++) {
      const uint32_t r = i * (64 / CW) + lane / CW;
      *(uint4 *)(wl + r * (16 * CW) + 16 * ((lane % CW) ^ turn(r))) = wd[i];
    }
#pragma unroll
    for (int i = 0; i < XI; i++) {
      const uint32_t b = i * (64 / CX) + lane / CX;
      if (b < XR) *(uint4 *)(xl + b * (16 * CX) + 16 * ((lane % CX) ^ (b & 7u))) = mv4_vector(xd[i]);
    }
    wave_order();
    uint32_t sc[(GPI + 1) / 2], zc[(GPI + 3) / 4];
#pragma unroll
    for (int k = 0; k < (GPI + 1) / 2; k++) sc[k] = sd[k];
#pragma unroll
    for (int k = 0; k < (GPI + 3) / 4; k++) zc[k] = zd[k];
    if (blk + NW < nblk) fetch(blk + NW);
#pragma unroll
    for (int u = 0; u < HB; u++) {
      uint4 xf[MT][4];
      f4 xs[MT][4 / GS];
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
        const uint32_t b = mt * 16 + n < XR ? mt * 16 + n : 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const uint32_t piece = 16 * u + (GS == 4 ? 4 * g + k : 4 * k + g);
          xf[mt][k] = *(const uint4 *)(xl + b * (16 * CX) + 16 * (piece ^ (b & 7u)));
        }
        if (ZP) {
#pragma unroll
          for (int k = 0; k < 4; k++) xs[mt][k / GS] = mv4_mfma<BF16>(xf[mt][k], ones, k % GS ? xs[mt][k / GS] : zero);
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; rt++) {
        const uint32_t r = rt * 16 + n;
        const uint4 w = *(const uint4 *)(wl + r * (16 * CW) + 16 * ((4 * u + g) ^ turn(r)));
        uint32_t d[4] = {w.x, w.y, w.z, w.w};
        if (GS < 4) mv4_transpose(d);
        f4 acc[MT];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const uint4 wf = mv4_codes<BF16>(d[k]);
#pragma unroll
          for (int mt = 0; mt < MT; mt++) acc[mt] = mv4_mfma<BF16>(xf[mt][k], wf, k % GS ? acc[mt] : zero);
          if (k % GS == GS - 1) {
            const int j = u * (4 / GS) + k / GS;
            const float s = f32_of_f16((uint16_t)(__shfl(sc[j / 2], (int)r) >> (16 * (j & 1))));
            const float z = ZP ? (float)(int8_t)(__shfl(zc[j / 4], (int)r) >> (8 * (j & 3))) : 0.0f;
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
              for (int i = 0; i < 4; i++)
                y[rt][mt][i] = fmaf(s, ZP ? fmaf(-z, xs[mt][k / GS][i], acc[mt][i]) : acc[mt][i], y[rt][mt][i]);
          }
        }
      }
    }
  }

  __syncthreads();
  float *red = (float *)lds;
#pragma unroll
  for (int rt = 0; rt < RT; rt++)
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int i = 0; i < 4; i++) red[((wave * RT + rt) * MT + mt) * 256 + i * 64 + lane] = y[rt][mt][i];
  __syncthreads();
  for (uint32_t k = threadIdx.x; k < RT * MT * 256; k += 64 * NW) {
    const uint32_t l = k & 63u, i = (k >> 6) & 3u, mt = (k >> 8) % MT, rt = (k >> 8) / MT;
    const uint32_t b = v0 + mt * 16 + 4 * (l >> 4) + i, r = r0 + rt * 16 + (l & 15u);
    if (b >= P.batch || b >= v0 + XR || r >= P.rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w++) v += red[w * RT * MT * 256 + k];
    store_as(P.y, b * P.y_stride + r, v, P.y_type);
  }
}

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
