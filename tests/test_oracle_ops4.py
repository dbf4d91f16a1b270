"""The 64-bit plain forms of the operators on 4-bit memory, pinned by worked
examples, closed forms and brute force on small sizes."""
import numpy as np
import pytest

from oracle import ops4


def test_gemv_worked_example():
    # codes 1 2 / 3 4, scale 0.5 and 0.25, zero points 1 and 2, x = (2, 10)
    packed = np.array([0x21, 0x43], np.uint8)
    s = np.array([0.5, 0.25], np.float16).view(np.uint16)
    y, a = ops4.gemv(packed, s, np.array([1, 2], np.int8), 2, 2, 2, np.array([[2.0, 10.0]]))
    assert y.tolist() == [[5.0, 5.5]]          # (0 * 2 + 1 * 10) / 2, (1 * 2 + 2 * 10) / 4
    assert a.tolist() == [[17.0, 17.5]]
    y, _ = ops4.gemv(packed, s, None, 2, 2, 2, np.array([[2.0, 10.0], [1.0, 0.0]]))
    assert y.tolist() == [[11.0, 11.5], [0.5, 0.75]]


@pytest.mark.parametrize("P", [32, 64, 128, 256])
@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (128, 32), (128, 128), (256, 64), (256, 256)])
def test_cache_places_cover_a_page_once(P, D, G):
    """Every nibble and every scale has one place, and together they fill the block."""
    seen = np.zeros(ops4.page_bytes(P, D, G) * 2, np.int64)
    for slot in range(P):
        for d in range(D):
            for at, sh in (ops4.k_place(P, D, d, slot), ops4.v_place(P, D, G, d, slot)):
                seen[2 * at + sh // 4] += 1
        for grp in range(D // G):
            for is_v in (False, True):
                at = ops4.scale_place(P, D, G, grp, slot, is_v)
                seen[2 * at:2 * at + 8] += 1
    assert np.all(seen == 1)


def test_cache_worked_places():
    # the layout read off its description: dword (g, c) has values 32 c + 8 g + 0..7
    assert ops4.k_place(64, 128, 0, 0) == (0, 0)
    assert ops4.k_place(64, 128, 1, 0) == (0, 4)
    assert ops4.k_place(64, 128, 32, 0) == (4, 0)       # g 0, c 1
    assert ops4.k_place(64, 128, 8, 0) == (16, 0)       # g 1, c 0
    assert ops4.k_place(64, 128, 127, 2) == (2 * 64 + 60 + 3, 4)
    base = 64 * 64 + 64 * 2 * 4
    assert ops4.v_place(64, 128, 64, 0, 0) == (base, 0)
    assert ops4.v_place(64, 128, 64, 16, 0) == (base, 4)
    assert ops4.v_place(64, 128, 64, 48, 1) == (base + 2 + 1, 4)
    assert ops4.v_place(64, 128, 64, 64, 0) == (base + 8, 0)       # h 1
    assert ops4.v_place(64, 128, 64, 1, 0) == (base + 16, 0)       # a 1
    assert ops4.v_place(64, 128, 64, 0, 4) == (base + 256, 0)      # g 1
    assert ops4.v_place(64, 128, 64, 0, 16) == (base + 1024, 0)    # tile 1


def test_put_then_get():
    rng = np.random.default_rng(5)
    P, D, G = 32, 128, 32
    block = rng.integers(0, 256, ops4.page_bytes(P, D, G)).astype(np.uint8)
    y = rng.standard_normal((2, D))
    c, s, m = ops4.quantize(y, G)
    ops4.put(block, P, D, G, 7, c[0], s[0], m[0], False)
    ops4.put(block, P, D, G, 7, c[1], s[1], m[1], True)
    k, v, sv = ops4.get(block, P, D, G, 7)
    for got, ref in ((k, y[0]), (v, y[1])):
        assert np.all(np.abs(got - ref) <= np.repeat((ref.reshape(-1, G).max(1) - ref.reshape(-1, G).min(1)) / 15, G) * 0.51
                      + 2 ** -11 * np.abs(ref).max())
    assert np.array_equal(sv, np.repeat(ops4.f64_from_bits(s[1]), G))


def test_quantize_worked_example_and_edges():
    y = np.array([[0.0, 1.0, 7.4, 15.0] + [3.0] * 28])
    c, s, m = ops4.quantize(y, 32)
    assert c[0, :5].tolist() == [0, 1, 7, 15, 3] and ops4.f64_from_bits(s).item() == 1.0 and m.item() == 0
    c, s, m = ops4.quantize(np.full((1, 32), -2.5), 32)        # one value: no step, the offset is the value
    assert not c.any() and s.item() == 0 and ops4.f64_from_bits(m).item() == -2.5
    c, s, m = ops4.quantize(np.array([[1e9] + [-1e9] * 31]), 32)   # held at fp16's ends
    assert ops4.f64_from_bits(m).item() == -65504 and c[0, 0] == 15 and not c[0, 1:].any()
    for x in (np.nan, np.inf, -np.inf):
        c, s, m = ops4.quantize(np.array([[x] + [1.0] * 31]), 32)
        assert not c.any() and s.item() == 0 and np.isnan(ops4.f64_from_bits(m).item())


def test_rotation_keeps_lengths_and_turns_pairs():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 64))
    a = rng.uniform(0, 6, (3, 16))
    for nb in (False, True):
        y = ops4.rotate(x, np.cos(a), np.sin(a), nb)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[:, 32:], x[:, 32:])
    e = np.zeros((1, 64))
    e[0, 3] = 1.0
    h = ops4.rotate(e, np.full((1, 16), 0.6), np.full((1, 16), 0.8), False)
    n = ops4.rotate(e, np.full((1, 16), 0.6), np.full((1, 16), 0.8), True)
    assert h[0, 3] == 0.6 and h[0, 19] == 0.8
    assert n[0, 3] == 0.6 and n[0, 2] == -0.8


def test_norm_closed_form():
    x = np.full((1, 64), 3.0)
    assert np.allclose(ops4.norm(x, np.full(64, 2.0), 0.0), 2.0)
    assert np.array_equal(ops4.norm(np.zeros((1, 64)), np.ones(64), 1e-6), np.zeros((1, 64)))


def test_attention_sees_what_the_masks_leave():
    assert ops4.visible(4, 0, 0) == [0, 1, 2, 3, 4]
    assert ops4.visible(6, 2, 0) == [5, 6]
    assert ops4.visible(6, 2, 3) == [0, 1, 2, 5, 6]
    assert ops4.visible(6, 9, 3) == list(range(7))
    assert ops4.visible(-1, 0, 4) == []
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((9, 64)), rng.standard_normal((9, 64))
    o, lse, _ = ops4.attention(np.zeros(64), k, v, np.ones((9, 64)), 1.0, 6, 2, 1)
    assert np.allclose(o, v[[0, 5, 6]].mean(0)) and np.isclose(lse, np.log(3))
    o, lse, _ = ops4.attention(100 * k[5] / np.linalg.norm(k[5]), k, v, np.ones((9, 64)), 100.0, 6, 2, 1)
    assert np.allclose(o, v[5])
    o, lse, _ = ops4.attention(k[0], k, v, np.ones((9, 64)), 1.0, -1, 0, 0)
    assert not o.any() and lse == -np.inf
