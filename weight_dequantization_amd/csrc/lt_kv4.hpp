// lt_kv4.hpp -- a paged key/value cache in 4 bits (gfx950, wave64): writing
// it, reading it back and attending to it.  The layout is lt_kv4_cache's.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lt_types.hpp"

namespace lt {

struct Kv4View {
  uint8_t *pages;
  uint64_t n_pages;
  uint32_t kv_heads, page_shift, dim, group;
  uint32_t block;            // bytes of one page and head
  uint32_t kc, sc;           // bytes of its codes (K or V) and of its scales (K or V)
};

struct Kv4Rows {
  const int32_t *q_start, *kv_len, *table;
  uint32_t n_seqs, max_pages, n_tokens;
};

__device__ __forceinline__ uint8_t *kv4_block(const Kv4View &C, uint32_t page, uint32_t head) {
  return C.pages + ((uint64_t)page * C.kv_heads + head) * C.block;
}

// byte offsets within a block
__device__ __forceinline__ uint32_t kv4_k_row(const Kv4View &C, uint32_t slot) { return slot * (C.dim / 2); }
__device__ __forceinline__ uint32_t kv4_scale(const Kv4View &C, uint32_t slot, uint32_t grp) {
  return ((grp << C.page_shift) + slot) * 4;
}
// unit (a, h) of token `slot`; 8 bytes hold the unit of 4 tokens
__device__ __forceinline__ uint32_t kv4_v_unit(const Kv4View &C, uint32_t slot, uint32_t a, uint32_t h) {
  return ((slot >> 2) * 16 + a) * (C.dim / 8) + h * 8 + (slot & 3) * 2;
}

struct Kv4Token {
  int32_t seq;               // -1: the row belongs to no sequence, or stands before position 0
  int32_t pos;
  int32_t page;              // -1: no valid page holds the position
};

// The sequence, position and page of row t, found by LV neighbouring lanes
// that ask for one row together (all 64 lanes take part).
template <int LV>
__device__ __forceinline__ Kv4Token kv4_token(const Kv4View &C, const Kv4Rows &B, uint32_t t, uint32_t j) {
  uint32_t cnt = 0;          // sequences that end at or before t
  for (uint32_t b = j; b < B.n_seqs; b += LV) cnt += (uint32_t)(B.q_start[b + 1] <= (int32_t)t);
#pragma unroll
  for (int d = 1; d < LV; d <<= 1) cnt += __shfl_xor(cnt, d);
  Kv4Token r{-1, 0, -1};
  if (t >= B.n_tokens || cnt >= B.n_seqs) return r;
  const int32_t first = B.q_start[cnt], last = B.q_start[cnt + 1];
  r.pos = B.kv_len[cnt] - (last - (int32_t)t);
  if (first > (int32_t)t || r.pos < 0) return r;
  r.seq = (int32_t)cnt;
  const uint32_t k = (uint32_t)r.pos >> C.page_shift;
  if (k < B.max_pages) {
    const int32_t p = B.table[(uint64_t)cnt * B.max_pages + k];
    if (p >= 0 && (uint64_t)p < C.n_pages) r.page = p;
  }
  return r;
}

// ------------------------------------------------------------------ append

struct Kv4NewRows {
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, o_ts, o_hs;
  const uint16_t *q_norm, *k_norm;
  const float *cos, *sin;
  const int32_t *positions;
  int32_t *status;
  uint32_t heads, rope_len, rotary, neighbours, bf16;   // heads: 0 without queries
  float eps;
};

__device__ __forceinline__ void load8(const uint16_t *p, bool bf16, float v[8]) {
  const uint4 d = *(const uint4 *)p;
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = f32_of_bits((uint16_t)(w[i >> 1] >> (16 * (i & 1))), bf16);
}

__device__ __forceinline__ void store8(uint16_t *p, bool bf16, const float v[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++)
    w[i] = (uint32_t)bits_of_f32(v[2 * i], bf16) | ((uint32_t)bits_of_f32(v[2 * i + 1], bf16) << 16);
  *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
}

// One head vector per LV = dim / 8 lanes, 8 neighbouring values a lane; a
// wave takes 64 / LV consecutive tokens of one head, so its K rows, its V
// units (4 tokens side by side) and its loads each fall together.  The
// rotation's products and sums are rounded one by one (no contraction), as
// its formula reads.
template <int LV>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4View C, Kv4Rows B, Kv4NewRows N) {
  constexpr uint32_t TPW = 64 / LV;
  const uint32_t lane = threadIdx.x & 63u, j = lane % LV;
  const uint32_t all = N.heads + 2 * C.kv_heads;
  const uint64_t w = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint32_t hd = (uint32_t)(w % all);
  const uint64_t t64 = w / all * TPW + lane / LV;
  const uint32_t t = t64 < B.n_tokens ? (uint32_t)t64 : B.n_tokens;   // n_tokens: no row
  const bool bf16 = N.bf16 != 0;
  Kv4Token k = kv4_token<LV>(C, B, t, j);
  const bool live = k.seq >= 0;
  int32_t row = k.pos;
  if (live && N.positions) row = N.positions[t];
  const bool turned = N.cos != nullptr;
  const bool bad = k.page < 0 || (turned && (row < 0 || (uint32_t)row >= N.rope_len));
  if (!live || bad) row = 0;

  const bool is_q = hd < N.heads, is_v = hd >= N.heads + C.kv_heads;
  const uint32_t h = is_q ? hd : is_v ? hd - N.heads - C.kv_heads : hd - N.heads;
  float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (live) {
    const uint16_t *src = is_q ? N.q + (int64_t)t * N.q_ts + (int64_t)h * N.q_hs
                               : is_v ? N.v + (int64_t)t * N.v_ts + (int64_t)h * N.v_hs
                                      : N.k + (int64_t)t * N.k_ts + (int64_t)h * N.k_hs;
    load8(src + 8 * j, bf16, y);
  }
  if (N.status && hd == N.heads && j == 0 && t < B.n_tokens)
    N.status[t] = live && bad ? LT_CHUNK_BAD_TABLE : LT_CHUNK_OK;

  if (!is_v) {
    const uint16_t *wt = is_q ? N.q_norm : N.k_norm;
    if (wt) {
      float ss = 0.0f, wv[8];
#pragma unroll
      for (int i = 0; i < 8; i++) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int d = 1; d < LV; d <<= 1) ss += __shfl_xor(ss, d);
      const float inv = rsqrtf(ss / (float)C.dim + N.eps);
      load8(wt + 8 * j, bf16, wv);
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = y[i] * inv * wv[i];
    }
    if (turned) {
      const uint32_t half = N.rotary / 2;
      const float *cr = N.cos + (uint64_t)row * half, *sr = N.sin + (uint64_t)row * half;
      if (N.neighbours) {
        if (8 * j < N.rotary) {
          const float4 c = *(const float4 *)(cr + 4 * j), s = *(const float4 *)(sr + 4 * j);
          const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const float a = y[2 * i], b = y[2 * i + 1];
            y[2 * i] = __fsub_rn(__fmul_rn(a, cv[i]), __fmul_rn(b, sv[i]));
            y[2 * i + 1] = __fadd_rn(__fmul_rn(b, cv[i]), __fmul_rn(a, sv[i]));
          }
        }
      } else {
        // the other value of each pair is rotary / 16 lanes away
        const bool second = 8 * j >= half, in = 8 * j < N.rotary;
        const uint32_t i0 = second ? 8 * j - half : 8 * j;
        const int other = (int)lane + (in ? (second ? -(int)(half / 8) : (int)(half / 8)) : 0);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = __shfl(y[i], other);
        if (in) {
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const float c = cr[i0 + i], s = sr[i0 + i];
            y[i] = second ? __fadd_rn(__fmul_rn(y[i], c), __fmul_rn(o[i], s))
                          : __fsub_rn(__fmul_rn(y[i], c), __fmul_rn(o[i], s));
          }
        }
      }
    }
  }
  if (is_q) {
    if (live) {
      if (bad) {
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __builtin_nanf("");
      }
      store8(N.q_out + (int64_t)t * N.o_ts + (int64_t)h * N.o_hs + 8 * j, bf16, y);
    }
    return;
  }

  // the group's range, over group / 8 lanes
  const uint32_t lg = C.group / 8;
  bool odd = false;
  float lo = __builtin_inff(), hi = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < 8; i++) {
    odd |= !(fabsf(y[i]) <= 3.402823466e38f);
    y[i] = fminf(fmaxf(y[i], -65504.0f), 65504.0f);
    lo = fminf(lo, y[i]);
    hi = fmaxf(hi, y[i]);
  }
  uint32_t oddv = odd;
  for (uint32_t d = 1; d < lg; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, (int)d));
    hi = fmaxf(hi, __shfl_xor(hi, (int)d));
    oddv |= __shfl_xor(oddv, (int)d);
  }
  uint16_t mb = f16_of_f32(lo), sb = f16_of_f32((hi - lo) / 15.0f);
  const float m = f32_of_f16(mb), s = f32_of_f16(sb);
  const float inv = s > 0.0f ? 1.0f / s : 0.0f;
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float c = fminf(fmaxf(rintf((y[i] - m) * inv), 0.0f), 15.0f);
    codes |= (uint32_t)c << (4 * i);
  }
  if (oddv) {
    codes = 0;
    sb = 0;
    mb = 0x7E00u;
  }
  const bool put = live && !bad;
  const uint32_t slot = (uint32_t)k.pos & ((1u << C.page_shift) - 1);
  uint8_t *blk = put ? kv4_block(C, (uint32_t)k.page, h) : nullptr;
  if (is_v) {
    // values 16 apart share a unit: the 4 lanes that hold them exchange
    // their codes, and lane n of them writes units 8 b + 2 n and + 1
    const uint32_t jj = j & 7, b = jj & 1, n = jj >> 1;
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; i++) d[i] = __shfl(codes, (int)((lane & ~7u) + 2 * i + b));
    if (put) {
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const uint32_t sh = 4 * (2 * n + e);
        uint32_t u = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) u |= ((d[i] >> sh) & 15u) << (4 * i);
        *(uint16_t *)(blk + C.kc + C.sc + kv4_v_unit(C, slot, 8 * b + 2 * n + e, j >> 3)) = (uint16_t)u;
      }
    }
    blk += C.kc + C.sc + C.kc;
  } else {
    if (put) *(uint32_t *)(blk + kv4_k_row(C, slot) + 4 * ((j & 3) * (C.dim / 32) + (j >> 2))) = codes;
    blk += C.kc;
  }
  if (put && j % lg == 0) *(uint32_t *)(blk + kv4_scale(C, slot, j / lg)) = (uint32_t)sb | ((uint32_t)mb << 16);
}

// -------------------------------------------------------------------- read

struct Kv4ReadRows {
  void *k, *v;
  int32_t *status;
  uint32_t type;
};

// As the append: LV lanes a head vector, 8 values a lane.
template <int LV>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4View C, Kv4Rows B, Kv4ReadRows R) {
  constexpr uint32_t TPW = 64 / LV;
  const uint32_t lane = threadIdx.x & 63u, j = lane % LV;
  const uint32_t all = 2 * C.kv_heads;
  const uint64_t w = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint32_t hd = (uint32_t)(w % all);
  const uint64_t t64 = w / all * TPW + lane / LV;
  const uint32_t t = t64 < B.n_tokens ? (uint32_t)t64 : B.n_tokens;
  const Kv4Token k = kv4_token<LV>(C, B, t, j);
  const bool live = k.seq >= 0, is_v = hd >= C.kv_heads;
  const uint32_t h = is_v ? hd - C.kv_heads : hd;
  if (R.status && hd == 0 && j == 0 && t < B.n_tokens)
    R.status[t] = live && k.page < 0 ? LT_CHUNK_BAD_TABLE : LT_CHUNK_OK;
  void *out = is_v ? R.v : R.k;
  if (!live || !out) return;
  float y[8];
  if (k.page < 0) {
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = __builtin_nanf("");
  } else {
    const uint32_t slot = (uint32_t)k.pos & ((1u << C.page_shift) - 1);
    const uint8_t *blk = kv4_block(C, (uint32_t)k.page, h);
    uint32_t codes = 0;
    if (is_v) {
      blk += C.kc + C.sc;
      const uint32_t jj = j & 7, n = jj >> 1;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const uint32_t u = *(const uint16_t *)(blk + kv4_v_unit(C, slot, 8 * (jj & 1) + e, j >> 3));
        codes |= ((u >> (4 * n)) & 15u) << (4 * e);
      }
    } else {
      codes = *(const uint32_t *)(blk + kv4_k_row(C, slot) + 4 * ((j & 3) * (C.dim / 32) + (j >> 2)));
    }
    const uint32_t sm = *(const uint32_t *)(blk + C.kc + kv4_scale(C, slot, j / (C.group / 8)));
    const float s = f32_of_f16((uint16_t)sm), m = f32_of_f16((uint16_t)(sm >> 16));
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = fmaf((float)((codes >> (4 * i)) & 15u), s, m);
  }
  const uint64_t at = ((uint64_t)t * C.kv_heads + h) * C.dim + 8 * j;
  if (R.type == LT_F32) {
    float4 *o = (float4 *)((float *)out + at);
    o[0] = make_float4(y[0], y[1], y[2], y[3]);
    o[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    store8((uint16_t *)out + at, R.type == LT_BF16, y);
  }
}

// --------------------------------------------------------------- attention

struct Kv4Attn {
  const uint16_t *q;
  uint16_t *out;
  float *lse;
  int64_t q_ts, q_hs, o_ts, o_hs;
  uint32_t heads, ratio, bf16, window, sinks, max_q;
  float scale;
};

// One wave per row and head, lane l holding values l, l + 64, ..; one token
// after another with the running maximum and sum of the softmax.
template <int DPL>
__global__ void __launch_bounds__(256) kv4_attention_kernel(Kv4View C, Kv4Rows B, Kv4Attn A) {
  const uint32_t lane = threadIdx.x & 63u;
  const uint64_t w = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint64_t t64 = w / A.heads;
  const uint32_t t = t64 < B.n_tokens ? (uint32_t)t64 : B.n_tokens;
  const uint32_t head = (uint32_t)(w % A.heads), h = head / A.ratio;
  const Kv4Token k = kv4_token<64>(C, B, t, lane);
  uint32_t cnt = 0;
  for (uint32_t b = lane; b < B.n_seqs; b += 64) cnt += (uint32_t)(B.q_start[b + 1] <= (int32_t)t);
  for (int d = 1; d < 64; d <<= 1) cnt += __shfl_xor(cnt, d);
  if (t >= B.n_tokens || cnt >= B.n_seqs) return;
  if (t - (uint32_t)B.q_start[cnt] >= A.max_q) return;
  const uint32_t n = k.seq >= 0 ? (uint32_t)k.pos + 1 : 0;
  const uint32_t lo = A.window && n > A.window ? n - A.window : 0;
  float q[DPL], o[DPL], top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
  for (int i = 0; i < DPL; i++) {
    q[i] = f32_of_bits(A.q[(int64_t)t * A.q_ts + (int64_t)head * A.q_hs + lane + 64 * i], A.bf16 != 0);
    o[i] = 0.0f;
  }
  for (uint32_t p = A.sinks > 0 || lo == 0 ? 0 : lo; p < n; p++) {
    if (p >= A.sinks && p < lo) p = lo;
    const uint32_t pi = p >> C.page_shift, slot = p & ((1u << C.page_shift) - 1);
    const int32_t page = pi < B.max_pages ? B.table[(uint64_t)cnt * B.max_pages + pi] : -1;
    if (page < 0 || (uint64_t)page >= C.n_pages) {
      sum = __builtin_nanf("");
      continue;
    }
    const uint8_t *blk = kv4_block(C, (uint32_t)page, h);
    float x = 0.0f, v[DPL];
#pragma unroll
    for (int i = 0; i < DPL; i++) {
      const uint32_t d = lane + 64 * i, g = d / C.group, j = d / 8;
      const uint32_t kb = blk[kv4_k_row(C, slot) + 4 * ((j & 3) * (C.dim / 32) + (j >> 2)) + (d & 7) / 2];
      const uint32_t vb = *(const uint16_t *)(blk + C.kc + C.sc + kv4_v_unit(C, slot, d & 15, d >> 6));
      const uint32_t ks = *(const uint32_t *)(blk + C.kc + kv4_scale(C, slot, g));
      const uint32_t vs = *(const uint32_t *)(blk + 2 * C.kc + C.sc + kv4_scale(C, slot, g));
      const float kd = fmaf((float)((kb >> (4 * (d & 1))) & 15u), f32_of_f16((uint16_t)ks), f32_of_f16((uint16_t)(ks >> 16)));
      v[i] = fmaf((float)((vb >> (4 * ((d >> 4) & 3))) & 15u), f32_of_f16((uint16_t)vs), f32_of_f16((uint16_t)(vs >> 16)));
      x = fmaf(q[i], kd, x);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    x *= A.scale;
    const float nt = fmaxf(top, x), a = nt > top ? __expf(top - nt) : 1.0f, e = __expf(x - nt);
    top = nt;
    sum = fmaf(sum, a, e);
#pragma unroll
    for (int i = 0; i < DPL; i++) o[i] = fmaf(o[i], a, e * v[i]);
  }
#pragma unroll
  for (int i = 0; i < DPL; i++)
    A.out[(int64_t)t * A.o_ts + (int64_t)head * A.o_hs + lane + 64 * i] =
        bits_of_f32(sum == 0.0f ? 0.0f : o[i] / sum, A.bf16 != 0);
  if (A.lse && lane == 0) A.lse[(uint64_t)t * A.heads + head] = sum == 0.0f ? -__builtin_inff() : top + logf(sum);
}

}  // namespace lt
