"""Refusals of the operators on 4-bit memory: the library checks its
arguments before any device work, so these need no GPU."""
import ctypes as C

import pytest

import weight_dequantization_amd as lt

A = 0x10000              # never dereferenced: validation fails first
INVALID, UNSUPPORTED, OK = lt.LT_ERR_INVALID_ARG, lt.LT_ERR_UNSUPPORTED, lt.LT_OK


def gemv(packed=A, scales=A, zp=None, rows=64, cols=256, group=128, x=A, xs=256, batch=2, xt=lt.F16, y=A, ys=64,
         yt=lt.F16):
    return lt.lib().lt_gemv_int4(packed, scales, zp, rows, cols, group, x, xs, batch, xt, y, ys, yt, None)


@pytest.mark.parametrize("kw", [
    dict(packed=None), dict(scales=None), dict(x=None), dict(y=None), dict(batch=0), dict(rows=0), dict(cols=0),
    dict(group=0), dict(group=96), dict(xs=255), dict(ys=63), dict(xt=lt.F32), dict(xt=7), dict(yt=3), dict(x=A + 1),
    dict(y=A + 1), dict(y=A + 2, yt=lt.F32), dict(scales=A + 1), dict(rows=1, cols=3, group=3, xs=3)])
def test_gemv_invalid(kw):
    assert gemv(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(batch=65), dict(rows=1 << 31, ys=1 << 31)])
def test_gemv_unsupported(kw):
    assert gemv(**kw) == UNSUPPORTED


def cache(pages=A, n=4, P=64, H=2, D=128, G=64):
    return lt._Kv4Cache(pages, n, P, H, D, G)


def batch(q_start=A, kv_len=A, table=A, seqs=2, width=3, tokens=2, q=1, kv=100):
    return lt._Kv4Batch(q_start, kv_len, table, seqs, width, tokens, q, kv)


def rows(**kw):
    d = dict(k=A, v=A, q=A, q_out=A, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128,
             q_token_stride=512, q_head_stride=128, q_out_token_stride=512, q_out_head_stride=128, q_norm=A, k_norm=A,
             cos=A, sin=A, positions=A, heads=4, rope_len=100, rotary_dim=128, neighbours=0, eps=1e-6, type=lt.F16)
    d.update(kw)
    return lt._Kv4New(**d)


def append(c, b, r, status=None):
    return lt.lib().lt_kv4_append(C.byref(c) if c else None, C.byref(b) if b else None, C.byref(r) if r else None,
                                  status, None)


def read(c, b, k=A, v=A, kind=lt.F16, status=None):
    return lt.lib().lt_kv4_read(C.byref(c) if c else None, C.byref(b) if b else None, k, v, kind, status, None)


def attention(c, b, q=A, qs=(1024, 128), heads=8, kind=lt.F16, scale=0.1, out=A, os_=(1024, 128), lse=None, ws=A,
              n=1 << 40):
    return lt.lib().lt_kv4_attention(C.byref(c) if c else None, C.byref(b) if b else None, q, *qs, heads, kind, scale, 0,
                                     0, out, *os_, lse, ws, n, None)


BAD_VIEWS = [
    (dict(pages=None), {}, INVALID), (dict(pages=A + 8), {}, INVALID), (dict(n=0), {}, INVALID),
    (dict(H=0), {}, INVALID), (dict(P=16), {}, UNSUPPORTED), (dict(P=48), {}, UNSUPPORTED),
    (dict(P=512), {}, UNSUPPORTED), (dict(D=96), {}, UNSUPPORTED), (dict(D=512), {}, UNSUPPORTED),
    (dict(G=16), {}, UNSUPPORTED), (dict(G=48), {}, UNSUPPORTED), (dict(D=64, G=128), {}, UNSUPPORTED),
    (dict(n=1 << 31), {}, UNSUPPORTED), (dict(H=1 << 16), {}, UNSUPPORTED),
    ({}, dict(q_start=None), INVALID), ({}, dict(kv_len=None), INVALID), ({}, dict(table=None), INVALID),
    ({}, dict(width=0), INVALID), ({}, dict(q_start=A + 2), INVALID), ({}, dict(table=A + 2), INVALID),
    ({}, dict(kv_len=A + 1), INVALID), ({}, dict(tokens=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("c,b,want", BAD_VIEWS)
def test_cache_and_batch_refused_by_all(c, b, want):
    assert append(cache(**c), batch(**b), rows()) == want
    assert read(cache(**c), batch(**b)) == want
    assert attention(cache(**c), batch(**b)) == want


def test_null_structs_refused():
    for c, b in ((None, batch()), (cache(), None)):
        assert append(c, b, rows()) == INVALID and read(c, b) == INVALID and attention(c, b) == INVALID
    assert append(cache(), batch(), None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 8), dict(k_token_stride=252), dict(v_head_stride=4),
    dict(q=None), dict(q_out=None), dict(heads=0), dict(q=A + 8), dict(q_out=A + 8), dict(q_head_stride=12),
    dict(q_out_token_stride=20), dict(q_norm=A + 8), dict(k_norm=A + 2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(cos=None), dict(sin=None), dict(cos=A + 8), dict(sin=A + 4), dict(rotary_dim=0), dict(rotary_dim=24),
    dict(rotary_dim=144), dict(rope_len=0), dict(positions=A + 2), dict(type=lt.F32), dict(type=9)])
def test_append_invalid(kw):
    assert append(cache(), batch(), rows(**kw)) == INVALID


def test_append_status_alignment():
    assert append(cache(), batch(), rows(), A + 2) == INVALID


@pytest.mark.parametrize("kw", [dict(k=None, v=None), dict(k=A + 8), dict(v=A + 4), dict(kind=3), dict(status=A + 1)])
def test_read_invalid(kw):
    assert read(cache(), batch(), **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(q=A + 8), dict(out=A + 2), dict(qs=(1020, 128)), dict(os_=(1024, 132)),
    dict(heads=0), dict(heads=7), dict(kind=lt.F32), dict(scale=float("inf")), dict(scale=float("nan")), dict(lse=A + 2)])
def test_attention_invalid(kw):
    assert attention(cache(), batch(), **kw) == INVALID


def test_nothing_to_do_is_fine():
    assert append(cache(), batch(tokens=0), rows()) == OK
    assert read(cache(), batch(tokens=0)) == OK
    assert attention(cache(), batch(tokens=0)) == OK
    assert attention(cache(), batch(q_start=None, kv_len=None, table=None, seqs=0, width=0)) == OK


def test_page_bytes():
    assert lt.kv4_page_bytes(64, 128, 64) == 64 * 128 + 2 * 64 * 2 * 4
    assert lt.kv4_page_bytes(32, 64, 32) == 32 * 64 + 2 * 32 * 2 * 4
    with pytest.raises(lt.LtError) as e:
        lt.kv4_page_bytes(64, 100, 50)
    assert e.value.status == UNSUPPORTED


def test_binding_refuses_wrong_tensors():
    import torch
    z = lambda *s, d=torch.float16: torch.zeros(*s, dtype=d)   # noqa: E731
    c = lt.Kv4Cache.empty(2, 32, 2, 64, 32, device="cpu")
    b = lt.Kv4Batch(z(2, d=torch.int32), z(1, d=torch.int32), z(1, 2, d=torch.int32), 3, 3, 3)
    k = z(3, 2, 64)
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, z(3, 2, 32), k)                        # wrong head size
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, k.transpose(0, 2).contiguous().transpose(0, 2), k)   # last dimension strided
    with pytest.raises(TypeError):
        lt.kv4_append(c, b, k, k.bfloat16())
    with pytest.raises(TypeError):
        lt.kv4_append(c, b, k.float(), k.float())
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, k, k, cos=z(4, 16, d=torch.float32))
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, k, k, cos=z(4, 16), sin=z(4, 16))
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, k, k, k_norm=z(32))
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, k, k, q_out=k)
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, k, k, status=z(2, d=torch.int32))
    with pytest.raises(ValueError):
        lt.kv4_append(c, b, k, k, positions=z(3, d=torch.int64))
    with pytest.raises(ValueError):
        lt.kv4_read(c, b, k=z(3, 2, 32))
    with pytest.raises(TypeError):
        lt.kv4_read(c, b, dtype=torch.int8)
    with pytest.raises(ValueError):
        lt.kv4_attention(c, b, z(2, 4, 64))                        # rows
    with pytest.raises(TypeError):
        lt.kv4_attention(c, b, z(3, 4, 64), out=z(3, 4, 64, d=torch.bfloat16))
    with pytest.raises(ValueError):
        lt.kv4_attention(c, b, z(3, 4, 64), lse=z(3, 4))
    with pytest.raises(ValueError):
        lt.kv4_read(lt.Kv4Cache(c.pages[:, :, :-16], 32, 2, 64, 32), b)   # pages of another size
    with pytest.raises(ValueError):
        lt.kv4_read(c, lt.Kv4Batch(z(2, d=torch.int64), b.kv_len, b.page_table, 3, 3, 3))
    with pytest.raises(ValueError):
        lt.gemv_int4(z(64, d=torch.uint8), z(1), None, (2, 64), 64, z(3, 32))
    with pytest.raises(ValueError):
        lt.gemv_int4(z(64, d=torch.uint8), z(1), None, (2, 64), 64, z(3, 64), y=z(3, 3))
    with pytest.raises(TypeError):
        lt.gemv_int4(z(64, d=torch.uint8), z(1), None, (2, 64), 64, z(3, 64, d=torch.float32))


@pytest.mark.parametrize("b,kw", [
    (dict(seqs=1 << 16), {}), ({}, dict(heads=65538)), (dict(tokens=1 << 30, q=1), dict(heads=8)),
    (dict(q=(1 << 31) - 1), dict(heads=4))])
def test_attention_beyond_its_grid(b, kw):
    """Sizes that its launches could not index are refused, not cut."""
    assert attention(cache(), batch(**b), **kw) == UNSUPPORTED
