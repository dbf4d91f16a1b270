"""Plain 64-bit forms of the operators on 4-bit memory (test infrastructure).

numpy only, one formula after another, sharing no code with the HIP library:

* gemv: y[b, r] = sum_c x[b, c] (q[r, c] - zp[g]) s[g], the group of element
  e = r * cols + c being e // group, codes two per byte, low nibble first.
* the paged cache: a page holds, per kv head, K codes, K scales, V codes and
  V scales; where each value of a token lies is written out index by index.
* quantization of a group y: m = fp16(min y), s = fp16((max y - min y) / 15),
  code = clamp(round((y - m) / s), 0, 15), the code c standing for s c + m.
* head norm x / sqrt(mean x^2 + eps) * w and rotation of pairs (a, b) to
  (a cos - b sin, b cos + a sin).
* attention: softmax over the visible positions of scale q . k, times v.
"""
from __future__ import annotations

import numpy as np


def f64_from_bits(bits, bf16=False):
    """fp16 or bf16 bit patterns (uint16) as float64, exactly."""
    bits = np.asarray(bits, np.uint16)
    if bf16:
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return bits.view(np.float16).astype(np.float64)


# --------------------------------------------------------------------- gemv

def gemv(packed, scales, zp, rows, cols, group, x):
    """(y, a): y [b, rows] in float64 for x float64 [b, cols], and a the sum of
    the absolute products with q and zp apart, which bounds what any order of
    summation of either form can lose."""
    e = np.arange(rows * cols, dtype=np.int64)
    q = ((np.asarray(packed, np.uint8)[e >> 1] >> (4 * (e & 1))) & 15).astype(np.float64)
    g = e // group
    s = f64_from_bits(scales)[g]
    z = np.zeros(e.size) if zp is None else np.asarray(zp, np.int8).astype(np.float64)[g]
    w = ((q - z) * s).reshape(rows, cols)
    most = ((q + np.abs(z)) * np.abs(s)).reshape(rows, cols)
    return x @ w.T, np.abs(x) @ most.T


# -------------------------------------------------------------------- cache

def page_bytes(P, D, G):
    return 2 * (P * D // 2 + P * (D // G) * 4)


def k_place(P, D, d, slot):
    """(byte offset within a page and head, shift) of value d of a key."""
    dword = (d % 32 // 8) * (D // 32) + d // 32
    return slot * (D // 2) + 4 * dword + d % 8 // 2, 4 * (d % 2)


def v_place(P, D, G, d, slot):
    h, a, n = d // 64, d % 16, d % 64 // 16
    unit = (((slot // 16 * 4 + slot % 16 // 4) * 16 + a) * (D // 64) + h) * 4 + slot % 4
    return P * D // 2 + P * (D // G) * 4 + 2 * unit + n // 2, 4 * (n % 2)


def scale_place(P, D, G, grp, slot, is_v):
    at = P * D // 2 + (P * (D // G) * 4 + P * D // 2 if is_v else 0)
    return at + 4 * (grp * P + slot)


def get(block, P, D, G, slot):
    """(k, v, s_v) of one token from a page and head's bytes: values in
    float64 and the value scales, [D] each."""
    d, out = np.arange(D), []
    for is_v in (False, True):
        at, sh = v_place(P, D, G, d, slot) if is_v else k_place(P, D, d, slot)
        c = ((block[at].astype(np.int64) >> sh) & 15).astype(np.float64)
        at = scale_place(P, D, G, d // G, slot, is_v)[:, None] + np.arange(4)
        sm = f64_from_bits(np.ascontiguousarray(block[at]).view(np.uint16))
        with np.errstate(invalid="ignore"):
            out.append((sm[:, 0] * c + sm[:, 1], sm[:, 0]))
    return out[0][0], out[1][0], out[1][1]


def put(block, P, D, G, slot, codes, s_bits, m_bits, is_v):
    """Codes [D] and scale, offset bits [D/G] of one token into a page and head's bytes."""
    at, sh = v_place(P, D, G, np.arange(D), slot) if is_v else k_place(P, D, np.arange(D), slot)
    for part, keep in ((0, 0xF0), (4, 0x0F)):
        i = at[sh == part]
        block[i] = (block[i] & keep) | (codes[sh == part] << part).astype(np.uint8)
    for grp in range(D // G):
        i = scale_place(P, D, G, grp, slot, is_v)
        block[i:i + 4] = np.array([s_bits[grp], m_bits[grp]], np.uint16).view(np.uint8)


def quantize(y, G, wide=np.float64):
    """(codes [n, D], s bits [n, NG], m bits) of y [n, D], computed in `wide`.
    In float32, with the reciprocal of s rounded first, every step is the one
    that the library states; in float64 it is the formula."""
    y = np.asarray(y, wide)
    n, D = y.shape
    y = y.reshape(n, D // G, G)
    odd = ~np.isfinite(y).all(-1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = np.clip(np.where(np.isfinite(y), y, 0), -65504, 65504).astype(wide)
        lo, hi = y.min(-1), y.max(-1)
        m = lo.astype(np.float16)
        s = ((hi - lo) / wide(15)).astype(np.float16)
        inv = np.where(s > 0, wide(1) / s.astype(wide), wide(0)).astype(wide)
        c = np.clip(np.rint((y - m.astype(wide)[..., None]) * inv[..., None]), 0, 15).astype(np.int64)
    sb, mb = s.view(np.uint16).copy(), m.view(np.uint16).copy()
    sb[odd], mb[odd] = 0, 0x7E00
    c[odd] = 0
    return c.reshape(n, D), sb, mb


def norm(x, w, eps):
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w


def rotate(x, cos, sin, neighbours):
    """x [..., D], cos and sin [..., r / 2] float64."""
    y = x.copy()
    h = cos.shape[-1]
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if neighbours else (slice(0, h), slice(h, 2 * h))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


# ---------------------------------------------------------------- attention

def visible(p, window, sinks):
    """The positions that a row at position p sees, in order."""
    return [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]


def attention(q, k, v, sv, scale, p, window, sinks):
    """One row q [D] at position p over k, v, sv [L, D] float64.  Returns
    (out, lse, spread): spread bounds what a relative error of 1 in every
    weight (times 8 steps of the code, the part of a value that a rounded
    weight multiplies) and in every score could do to an element."""
    D = q.size
    j = visible(p, window, sinks)
    if not j:
        return np.zeros(D), -np.inf, (np.zeros(D), np.zeros(D))
    x = scale * (k[j] @ q)
    top = x.max()
    e = np.exp(x - top)
    w = e / e.sum()
    size = np.abs(scale) * (np.abs(k[j]) @ np.abs(q)).max()
    o = w @ v[j]
    return o, top + np.log(e.sum()), (w @ (8 * sv[j]), size * (w @ np.abs(v[j] - o)))
