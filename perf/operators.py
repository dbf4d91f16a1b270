"""The operators of a serving step on 4-bit memory, as cases to be measured.

gemv       y = x W^T with W held as packed INT4 codes, fp16 scales and int8
           zero points per group (the layout of dequant_int4), 1 to 64 rows x
append     new keys and values (and the queries beside them): norm of every
           head, position rotation, 4-bit quantization, into a paged cache
read       tokens of the cache back as the values that they stand for
attention  softmax(scale q K^T) V over the cache: single tokens, chunks,
           ragged lengths, a sliding window with first tokens kept visible

`own` False computes each in elementary torch operations in fp32, True calls
weight_dequantization_amd.  Both take what prepare() returns.

The cache.  One uint8 tensor [pages, kv_heads, bytes of a page and head]; for
P tokens a page, head size D, groups of G values (NG = D / G a head), a page
and head holds in order
  K codes   [P][4][D/32] dwords: dword (g, c) has dims 32 c + 8 g + 0..7,
            low nibble first
  K scales  [NG][P] pairs of fp16 (s, m): a code c stands for s c + m
  V codes   [P/16][4][16][D/64][4] 16-bit units: unit (tile, g, a, h, i) has
            dims 64 h + a + 0, 16, 32, 48 of token 16 tile + 4 g + i
  V scales  [NG][P] pairs (s, m)
Quantization of a group y: m = fp16(min y), s = fp16((max y - min y) / 15),
code = clamp(round((y - m) (1 / s)), 0, 15), 0 where s is 0.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # ---- matrix-vector products
        # the smallest weight of this repository's configurations, one token: latency
        dict(name="gemv 1024x1024 one token", op="gemv", rows=1024, cols=1024, group=256, batch=1, zp=True,
             dtype="fp16", out="fp16"),
        # the MLP projection that the repository's headline decodes, one token: bandwidth
        dict(name="gemv 8192x28672 one token", op="gemv", rows=8192, cols=28672, group=128, batch=1, zp=True,
             dtype="fp16", out="fp16"),
        # a ragged projection with fine groups for a small batch of tokens
        dict(name="gemv 4999x8160 13 tokens", op="gemv", rows=4999, cols=8160, group=32, batch=13, zp=True,
             dtype="bf16", out="bf16"),
        # ---- writing the cache
        # one token of 64 sequences, the heads of a 70B-shaped layer (8192 = 64 x 128 and 1024 = 8 x 128)
        dict(name="append 64 single tokens", op="append", seqs=64, q_most=1, q_least=1, kv_least=1, kv_most=4096,
             heads=64, kv_heads=8, dim=128, group=64, page=64, dtype="fp16", norm=True, rotary=128, pairs="half"),
        # prompts of several lengths written at once
        dict(name="append ragged prompts", op="append", seqs=5, q_most=3500, q_least=1, kv_least=1, kv_most=3500,
             heads=32, kv_heads=8, dim=128, group=64, page=64, dtype="bf16", norm=True, rotary=64, pairs="neighbours"),
        # ---- reading it back
        # a short tail of one sequence, small heads
        dict(name="read 37 tokens", op="read", seqs=1, q_most=37, q_least=37, kv_least=37, kv_most=37, kv_heads=4,
             dim=64, group=32, page=32, dtype="bf16"),
        # whole prefixes, as for a hand-over to code that wants dense keys and values
        dict(name="read 16 prefixes", op="read", seqs=16, q_most=8192, q_least=100, kv_least=100, kv_most=8192,
             kv_heads=8, dim=128, group=64, page=64, dtype="fp16"),
        # ---- attention
        # one sequence early in its answer: latency
        dict(name="attention 1 token of 333", op="attention", seqs=1, q_most=1, q_least=1, kv_least=333, kv_most=333,
             heads=64, kv_heads=8, dim=128, group=64, page=64, dtype="fp16", window=0, sinks=0),
        # an ordinary serving batch: bandwidth
        dict(name="attention 64 ragged", op="attention", seqs=64, q_most=1, q_least=1, kv_least=500, kv_most=16384,
             heads=64, kv_heads=8, dim=128, group=64, page=64, dtype="bf16", window=0, sinks=0),
        # one long context
        dict(name="attention 1 token of 131071", op="attention", seqs=1, q_most=1, q_least=1, kv_least=131071,
             kv_most=131071, heads=64, kv_heads=8, dim=128, group=64, page=64, dtype="fp16", window=0, sinks=0),
        # chunks of prompts over what is cached already: arithmetic
        dict(name="attention prompt chunks", op="attention", seqs=2, q_most=2048, q_least=1531, kv_least=4000,
             kv_most=5000, heads=64, kv_heads=8, dim=128, group=128, page=128, dtype="bf16", window=0, sinks=0),
        # four drafted tokens a sequence, a window with the first tokens kept, odd head ratio, some
        # sequences shorter than the draft (rows that see nothing)
        dict(name="attention window, 4 drafted", op="attention", seqs=16, q_most=4, q_least=4, kv_least=2,
             kv_most=20000, heads=24, kv_heads=8, dim=64, group=32, page=32, dtype="fp16", window=4096, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemv", "append", "read", "attention", "attention"))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "gemv":
        group = rng.choice((32, 64, 128, 256))
        cols = group * max(1, _log(rng, 512, 28672) // group)
        return dict(op=op, rows=_log(rng, 100, 8192), cols=cols, group=group, batch=_log(rng, 1, 32),
                    zp=rng.random() < 0.75, dtype=dtype, out=rng.choice((dtype, dtype, "fp32")))
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    c = dict(op=op, kv_heads=kv_heads, dim=dim, group=rng.choice((32, 64)), page=rng.choice((32, 64, 128)),
             dtype=dtype)
    if op == "append":
        most = _log(rng, 1, 2000)
        return dict(c, seqs=rng.randint(1, 6), q_most=most, q_least=rng.randint(0, most), kv_least=1,
                    kv_most=most + _log(rng, 1, 1000), heads=kv_heads * rng.choice((1, 2, 3, 8)),
                    norm=rng.random() < 0.6, rotary=rng.choice((0, 32, dim)),
                    pairs=rng.choice(("half", "neighbours")))
    if op == "read":
        most = _log(rng, 20, 6000)
        return dict(c, seqs=rng.randint(1, 8), q_most=most, q_least=rng.randint(1, most), kv_least=most,
                    kv_most=most + rng.randint(0, 500))
    c.update(group=rng.choice((32, 64, dim if dim < 256 else 128)), heads=kv_heads * rng.choice((1, 2, 4, 5, 8)))
    window = rng.choice((0, 0, _log(rng, 16, 4096)))
    c.update(window=window, sinks=rng.randint(0, 9) if window else 0)
    if rng.random() < 0.6:   # single tokens and drafts
        q = rng.choice((1, 1, 1, rng.randint(2, 8)))
        most = _log(rng, 64, 30000)
        return dict(c, seqs=max(1, min(64, _log(rng, 1, 64), 250000 // most)), q_most=q, q_least=q,
                    kv_least=rng.randint(1, most), kv_most=most)
    q = _log(rng, 16, 1024)
    return dict(c, seqs=rng.randint(1, 3 if dim < 256 else 1), q_most=q, q_least=rng.randint(1, q), kv_least=q,
                kv_most=q + _log(rng, 16, 3000))


def _lengths(case):
    """Host lengths of a case's sequences, from the case alone: (query lengths, cache lengths after the new tokens)."""
    n = case["seqs"]
    g = torch.Generator().manual_seed(n * 7919 + case["kv_most"] * 31 + case["q_most"])
    kv = torch.randint(case["kv_least"], case["kv_most"] + 1, (n,), generator=g)
    kv[0] = case["kv_most"]
    q = torch.randint(case["q_least"], case["q_most"] + 1, (n,), generator=g)
    q[0] = case["q_most"]
    if n > 1 and case["op"] == "attention":
        kv[-1] = case["kv_least"]
    if case["op"] != "attention":
        kv = torch.maximum(kv, q)
    return q, kv


# ------------------------------------------------------------- what is at hand

def _page_bytes(P, D, G):
    return P * D + 2 * P * (D // G) * 4


def _places(pages, P, D, G):
    """Views of the four parts of a cache: K codes as bytes [n, H, P, 4, D/32, 4], K scales [n, H, NG, P, 2] fp16,
    V codes as bytes [n, H, P/16, 4, 16, D/64, 4, 2], V scales as the K scales."""
    n, H, _ = pages.shape
    kc, sc, NG = P * D // 2, P * (D // G) * 4, D // G
    return (pages[:, :, :kc].view(n, H, P, 4, D // 32, 4),
            pages[:, :, kc:kc + sc].view(torch.float16).view(n, H, NG, P, 2),
            pages[:, :, kc + sc:2 * kc + sc].view(n, H, P // 16, 4, 16, D // 64, 4, 2),
            pages[:, :, 2 * kc + sc:].view(torch.float16).view(n, H, NG, P, 2))


def _quantize(y, G):
    """Codes (as fp32 whole numbers) [T, H, D] and (s, m) [T, H, NG, 2] fp16 of fp32 y [T, H, D]."""
    T, H, D = y.shape
    y = y.reshape(T, H, D // G, G)
    lo, hi = y.amin(-1), y.amax(-1)
    m = lo.to(torch.float16)
    s = ((hi - lo) / 15.0).to(torch.float16)
    inv = torch.where(s > 0, 1.0 / s.float(), torch.zeros_like(lo))
    codes = torch.round((y - m.float()[..., None]) * inv[..., None]).clamp(0, 15)
    return codes.reshape(T, H, D), torch.stack((s, m), -1)


def _store(pages, P, D, G, page, slot, kq, ks, vq, vs):
    """Codes [T, H, D] and scales [T, H, NG, 2] of T tokens at (page, slot)."""
    T, H, _ = kq.shape
    Kc, Ks, Vc, Vs = _places(pages, P, D, G)
    k = kq.to(torch.uint8).reshape(T, H, D // 32, 4, 4, 2).transpose(2, 3)
    Kc[page, :, slot] = k[..., 0] | (k[..., 1] << 4)
    v = vq.to(torch.uint8).reshape(T, H, D // 64, 2, 2, 16).permute(0, 1, 5, 2, 3, 4)
    Vc[page, :, slot // 16, slot % 16 // 4, :, :, slot % 4] = v[..., 0] | (v[..., 1] << 4)
    Ks[page, :, :, slot] = ks
    Vs[page, :, :, slot] = vs


def _values(pages, P, D, G, page, slot):
    """K and V values in fp32 [T, H, D] of the tokens at (page, slot)."""
    T, H = page.shape[0], pages.shape[1]
    Kc, Ks, Vc, Vs = _places(pages, P, D, G)
    b = Kc[page, :, slot]                                              # [T, H, 4, D/32, 4]
    k = torch.stack((b & 15, b >> 4), -1).transpose(2, 3).reshape(T, H, D // G, G).float()
    b = Vc[page, :, slot // 16, slot % 16 // 4, :, :, slot % 4]        # [T, H, 16, D/64, 2]
    v = torch.stack((b & 15, b >> 4), -1).permute(0, 1, 3, 4, 5, 2).reshape(T, H, D // G, G).float()
    ks, vs = Ks[page, :, :, slot].float(), Vs[page, :, :, slot].float()   # [T, H, NG, 2]
    k = k * ks[..., :1] + ks[..., 1:]
    v = v * vs[..., :1] + vs[..., 1:]
    return k.reshape(T, H, D), v.reshape(T, H, D)


def _keys_and_values(n, H, D, g):
    """Keys with channels of their own mean and width, values around zero."""
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    return r(n, H, D) * (0.7 + 0.3 * r(1, H, D).abs()) + 0.5 * r(1, H, D), r(n, H, D)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)   # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    dt = TYPES[case["dtype"]]
    if case["op"] == "gemv":
        rows, cols, G = case["rows"], case["cols"], case["group"]
        q = torch.round(randn(rows * cols // 2, 2) * 3 + 7.5).clamp_(0, 15).to(torch.uint8)
        return dict(case=case, packed=q[:, 0] | (q[:, 1] << 4),
                    scales=(rand(rows * cols // G) * 0.045 + 0.005).to(torch.float16),
                    zp=(rand(rows * cols // G) * 16).to(torch.int8) if case["zp"] else None,
                    x=randn(case["batch"], cols).to(dt))
    P, D, G, H = case["page"], case["dim"], case["group"], case["kv_heads"]
    q_len, kv_len = _lengths(case)
    n, T = case["seqs"], int(q_len.sum())
    need = [-(-int(x) // P) for x in kv_len]
    total, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    s = dict(case=case, q_start=torch.cat((torch.zeros(1, dtype=torch.int64), q_len.cumsum(0))).to(DEV, torch.int32),
             kv_len=kv_len.to(DEV, torch.int32), table=table.to(DEV), tokens=T, q_most=int(q_len.max()),
             kv_most=int(kv_len.max()))
    # what earlier owners left in the pages, then the tokens that are cached already
    s["pages"] = torch.randint(0, 256, (total, H, _page_bytes(P, D, G)), generator=g, device=DEV, dtype=torch.uint8)
    have = kv_len - q_len if case["op"] == "append" else kv_len
    seq = torch.repeat_interleave(torch.arange(n), have)
    pos = torch.cat([torch.arange(int(x)) for x in have]) if len(have) else seq
    page, slot = table[seq, pos // P].long().to(DEV), (pos % P).to(DEV)
    for a in range(0, len(seq), 1 << 17):
        p, o = page[a:a + (1 << 17)], slot[a:a + (1 << 17)]
        k, v = _keys_and_values(len(p), H, D, g)
        _store(s["pages"], P, D, G, p, o, *_quantize(k, G), *_quantize(v, G))
    if case["op"] == "append":
        k, v = _keys_and_values(T, H, D, g)
        hq = case["heads"]
        # one projection's output, as it leaves the layer before
        s["qkv"] = torch.cat((randn(T, hq, D), k, v), 1).to(dt)
        if case["norm"]:
            s["q_norm"], s["k_norm"] = ((0.9 + 0.2 * rand(D)).to(dt) for _ in range(2))
        if case["rotary"]:
            r = case["rotary"]
            f = 10000.0 ** (-torch.arange(0, r, 2, device=DEV).double() / r)
            a = torch.arange(s["kv_most"], device=DEV).double()[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
    if case["op"] == "attention":
        s["q"] = (1.5 * randn(T, case["heads"], D)).to(dt)
    return s


# ------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["op"]](state, case)


def _tokens(state, case):
    """(sequence, position in its cache, page, slot) of each new token."""
    qs = state["q_start"].long()
    t = torch.arange(state["tokens"], device=DEV)
    seq = torch.searchsorted(qs[1:], t, right=True)
    pos = state["kv_len"].long()[seq] - (qs[1:] - qs[:-1])[seq] + t - qs[seq]
    return seq, pos, state["table"][seq, pos // case["page"]].long(), pos % case["page"]


def _plain_gemv(state, case):
    rows, cols, G = case["rows"], case["cols"], case["group"]
    p = state["packed"]
    w = torch.stack((p & 15, p >> 4), -1).reshape(-1, G).float()
    if state["zp"] is not None:
        w = w - state["zp"].float()[:, None]
    w = (w * state["scales"].float()[:, None]).reshape(rows, cols)
    return (state["x"].float() @ w.t()).to(TYPES[case["out"]])


def _norm(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()


def _rotate(x, cos, sin, pairs):
    r = 2 * cos.shape[-1]
    y, rest = x[..., :r], x[..., r:]
    cos, sin = cos[:, None], sin[:, None]
    if pairs == "half":
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((y, rest), -1)


def _plain_append(state, case):
    P, D, G, hq, H = case["page"], case["dim"], case["group"], case["heads"], case["kv_heads"]
    dt = TYPES[case["dtype"]]
    _, pos, page, slot = _tokens(state, case)
    q, k, v = state["qkv"].float().split((hq, H, H), 1)
    if case["norm"]:
        q, k = _norm(q, state["q_norm"]), _norm(k, state["k_norm"])
    if case["rotary"]:
        cos, sin = state["cos"][pos], state["sin"][pos]
        q, k = _rotate(q, cos, sin, case["pairs"]), _rotate(k, cos, sin, case["pairs"])
    _store(state["pages"], P, D, G, page, slot, *_quantize(k, G), *_quantize(v, G))
    k, v = _values(state["pages"], P, D, G, page, slot)
    return dict(q=q.to(dt), k=k.to(dt), v=v.to(dt))


def _plain_read(state, case):
    _, _, page, slot = _tokens(state, case)
    k, v = _values(state["pages"], case["page"], case["dim"], case["group"], page, slot)
    return dict(k=k.to(TYPES[case["dtype"]]), v=v.to(TYPES[case["dtype"]]))


def _plain_attention(state, case):
    P, D, G, hq, H = case["page"], case["dim"], case["group"], case["heads"], case["kv_heads"]
    n, Q, L, R = case["seqs"], state["q_most"], state["kv_most"], hq // H
    seq, pos, _, _ = _tokens(state, case)
    row = torch.arange(state["tokens"], device=DEV) - state["q_start"].long()[seq]
    q = torch.zeros(n, Q, hq, D, device=DEV)
    q[seq, row] = state["q"].float()
    at = torch.full((n, Q), -1, dtype=torch.int64, device=DEV)   # the position of each row, -1 where there is none
    at[seq, row] = pos
    j = torch.arange(L, device=DEV)
    there = j < state["kv_len"][:, None]                         # [n, L]
    page = torch.where(there, state["table"][:, j // P], 0).long().reshape(-1)
    k, v = _values(state["pages"], P, D, G, page, (j % P).repeat(n))
    there = there.reshape(-1, 1, 1)
    k = torch.where(there, k, 0.0).reshape(n, L, H, D).permute(0, 2, 3, 1)
    v = torch.where(there, v, 0.0).reshape(n, L, H, D).permute(0, 2, 1, 3)
    q = q.reshape(n, Q, H, R, D).permute(0, 2, 1, 3, 4).reshape(n, H, Q * R, D)
    x = torch.matmul(q, k) * D ** -0.5
    seen = j <= at[..., None]
    if case["window"]:
        seen &= (j > at[..., None] - case["window"]) | (j < case["sinks"])
    seen = seen[:, None, :, None].expand(n, 1, Q, R, L).reshape(n, 1, Q * R, L)
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total > 0, total, 1.0)
    o = o.reshape(n, H, Q, R, D).permute(0, 2, 1, 3, 4).reshape(n, Q, hq, D)
    return o[seq, row].to(TYPES[case["dtype"]])


def _cache(lt, state, case):
    return (lt.Kv4Cache(state["pages"], case["page"], case["kv_heads"], case["dim"], case["group"]),
            lt.Kv4Batch(state["q_start"], state["kv_len"], state["table"], state["tokens"], state["q_most"],
                        state["kv_most"]))


def _own_gemv(state, case):
    import weight_dequantization_amd as lt
    return lt.gemv_int4(state["packed"], state["scales"], state["zp"], (case["rows"], case["cols"]), case["group"],
                        state["x"], dtype=TYPES[case["out"]])


def _own_append(state, case):
    import weight_dequantization_amd as lt
    cache, batch = _cache(lt, state, case)
    hq, H = case["heads"], case["kv_heads"]
    qkv = state["qkv"]
    q = lt.kv4_append(cache, batch, qkv[:, hq:hq + H], qkv[:, hq + H:], q=qkv[:, :hq], q_norm=state.get("q_norm"),
                      k_norm=state.get("k_norm"), eps=1e-6, cos=state.get("cos"), sin=state.get("sin"),
                      neighbours=case["pairs"] == "neighbours")
    k, v = lt.kv4_read(cache, batch, dtype=TYPES[case["dtype"]])
    return dict(q=q, k=k, v=v)


def _own_read(state, case):
    import weight_dequantization_amd as lt
    k, v = lt.kv4_read(*_cache(lt, state, case), dtype=TYPES[case["dtype"]])
    return dict(k=k, v=v)


def _own_attention(state, case):
    import weight_dequantization_amd as lt
    return lt.kv4_attention(*_cache(lt, state, case), state["q"], scale=case["dim"] ** -0.5, window=case["window"],
                            sinks=case["sinks"])


_plain = dict(gemv=_plain_gemv, append=_plain_append, read=_plain_read, attention=_plain_attention)
_own = dict(gemv=_own_gemv, append=_own_append, read=_own_read, attention=_own_attention)


# ----------------------------------------------------------- what a pass needs

def _seen(lo, hi, window, sinks):
    """Tokens that rows at positions lo .. hi - 1 see: (in all, by any of them)."""
    lo = max(lo, 0)
    if hi <= lo:
        return 0, 0
    total = 0
    for p in range(lo, hi):
        near = p + 1 if not window else min(window, p + 1)
        total += near + min(sinks, p + 1 - near)
    first = 0 if not window else max(0, lo + 1 - window)
    return total, hi - first + min(sinks, first)


def work(case):
    if case["op"] == "gemv":
        rows, cols, b = case["rows"], case["cols"], case["batch"]
        groups = rows * cols // case["group"]
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": rows * cols // 2 + groups * (3 if case["zp"] else 2) + b * cols * 2 + b * rows * out,
                "flops": 2 * rows * cols * b}
    q_len, kv_len = (x.tolist() for x in _lengths(case))
    D, H = case["dim"], case["kv_heads"]
    token = H * (D + 2 * (D // case["group"]) * 4)   # a token's keys and values in the cache
    T = sum(q_len)
    if case["op"] == "read":
        return {"bytes": T * (token + 4 * H * D), "flops": 4 * T * H * D}
    if case["op"] == "append":   # inputs and queries, the cache written and read back, the values
        hq = case["heads"]
        tables = 4 * case["rotary"] * len({p for a, b in zip(q_len, kv_len) for p in range(b - a, b)})
        return {"bytes": T * ((hq + 2 * H) * D * 2 + hq * D * 2 + 2 * token + 4 * H * D) + tables,
                "flops": T * (hq + 2 * H) * D * 10}
    hq, flops, bytes_ = case["heads"], 0, 0
    for a, b in zip(q_len, kv_len):
        total, union = _seen(b - a, b, case["window"], case["sinks"])
        flops += 4 * D * hq * total
        bytes_ += union * token + 4 * a * hq * D
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------- in 64 bits, for itself

def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "gemv":
        n = case["rows"] * case["cols"]
        at = torch.arange(n // 2, device=DEV)
        q = torch.zeros(n, dtype=d, device=DEV)
        q[2 * at] = s["packed"].remainder(16).to(d)
        q[2 * at + 1] = torch.div(s["packed"], 16, rounding_mode="floor").to(d)
        q = q.view(-1, case["group"])
        if s["zp"] is not None:
            q -= s["zp"].to(d).unsqueeze(1)
        q *= s["scales"].to(d).unsqueeze(1)
        return (q.view(case["rows"], case["cols"]) @ s["x"].to(d).t()).t().contiguous()
    q_len, kv_len = (x.tolist() for x in _lengths(case))
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        # the cache stands for the keys and values themselves; what is left is the error of the 4 bits, which
        # says something where the groups are small and many
        pos = torch.cat([torch.arange(b - a, b) for a, b in zip(q_len, kv_len)]).to(DEV)
        x = s["qkv"].to(d)
        hq = case["heads"]
        q, k, v = x[:, :hq].clone(), x[:, hq:hq + H].clone(), x[:, hq + H:]
        for y, w in ((q, "q_norm"), (k, "k_norm")):
            if case["norm"]:
                y /= ((y ** 2).sum(-1, keepdim=True) / D + 1e-6) ** 0.5
                y *= s[w].to(d)
            r = case["rotary"]
            for i in range(r // 2):
                a, b = (i, i + r // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
                turn = torch.complex(s["cos"][pos, i].to(d), s["sin"][pos, i].to(d))
                z = torch.complex(y[:, :, a], y[:, :, b]) * turn[:, None]
                y[:, :, a], y[:, :, b] = z.real, z.imag
        near = case["group"] <= 64 and k.numel() >= 500 * case["group"]
        return dict(q=q, k=k if near else None, v=v if near else None)

    def nibbles(b):   # bytes [..., n] to codes [..., 2 n]
        return torch.cat((b.remainder(16).unsqueeze(-1), torch.div(b, 16, rounding_mode="floor").unsqueeze(-1)),
                         -1).flatten(-2).to(d)

    def tokens(i, h, first, last):
        """K and V of positions first .. last - 1 of sequence i, head h: whole pages, unpacked tile by tile."""
        if last <= first:
            return torch.zeros(2, 0, D, dtype=d, device=DEV)
        pages = s["table"][i, first // P:-(-last // P)].long()
        raw = s["pages"][pages, h]
        code, scale, groups = P * D // 2, P * (D // case["group"]) * 4, D // case["group"]
        k = nibbles(raw[:, :code].reshape(-1, 4, D // 32, 4)).permute(0, 2, 1, 3).reshape(len(pages) * P, D)
        v = nibbles(raw[:, code + scale:2 * code + scale].reshape(-1, P // 16, 4, 16, D // 64, 4, 2))
        v = v.permute(0, 1, 2, 5, 4, 6, 3).reshape(len(pages) * P, D)   # page, tile, g, i, h, dims / 16, a
        both = []
        for codes, at in ((k, code), (v, 2 * code + scale)):
            sm = raw[:, at:at + scale].contiguous().view(torch.float16).view(-1, groups, P, 2).to(d)
            sm = sm.transpose(1, 2).reshape(-1, groups, 1, 2)
            both.append((codes.view(-1, groups, case["group"]) * sm[..., 0] + sm[..., 1]).view(-1, D))
        off = first // P * P
        return torch.stack(both)[:, first - off:last - off]

    if case["op"] == "read":
        both = [torch.stack([tokens(i, h, b - a, b) for h in range(H)], 2)
                for i, (a, b) in enumerate(zip(q_len, kv_len))]
        both = torch.cat(both, 1)
        return dict(k=both[0], v=both[1])
    R = case["heads"] // H
    out = torch.zeros(sum(q_len), case["heads"], D, dtype=d, device=DEV)
    start = 0
    for i, (a, b) in enumerate(zip(q_len, kv_len)):
        for h in range(H):
            k, v = tokens(i, h, 0, b)
            for r in range(R * (a > 0)):
                x = s["q"][start:start + a, h * R + r].to(d) @ k.t() / math.sqrt(D)
                p = torch.arange(b - a, b, device=DEV).unsqueeze(1)
                j = torch.arange(b, device=DEV).unsqueeze(0)
                hidden = j > p
                if case["window"]:
                    hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
                w = torch.softmax(x.masked_fill(hidden, -math.inf), 1).nan_to_num(0.0)   # a row that sees nothing: 0
                out[start:start + a, h * R + r] = w @ v
        start += a
    return out
