"""Products of a few vectors with INT4 matrices (gemv_int4) against the
64-bit form.

Tolerance.  Products of a code with a 16-bit value are exact in fp32.  The
sum over cols terms of row r is taken in partial sums: chains of at most 160
terms (one matrix-core step of 128, with the joins of waves and lanes), then a
chain of at most cols / 32 partial sums.  Each rounding loses at most 2^-24 of
a partial sum that is at most sum |x| (q + |zp|) s, codes and zero points
apart.  Then y is rounded once to its type (half a unit in the last place,
and fp16's smallest step)."""
import numpy as np
import pytest
import torch

import weight_dequantization_amd as lt
from oracle import ops4

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield
    torch.cuda.synchronize()


def make(rows, cols, group, batch, dtype, zp=True, seed=0):
    rng = np.random.default_rng(seed + rows * 7 + cols * 3 + batch)
    packed = rng.integers(0, 256, rows * cols // 2).astype(np.uint8)
    n = rows * cols // group
    scales = rng.uniform(0.005, 0.05, n).astype(np.float16)
    z = rng.integers(0, 16, n).astype(np.int8) if zp else None
    x = torch.from_numpy(rng.standard_normal((batch, cols))).to(dtype)
    return packed, scales, z, x


def dev(packed, scales, z):
    return (torch.from_numpy(packed).to(DEV), torch.from_numpy(scales).to(DEV),
            None if z is None else torch.from_numpy(z).to(DEV))


def check(y, packed, scales, z, rows, cols, group, x, out):
    ref, a = ops4.gemv(packed, scales.view(np.uint16), z, rows, cols, group, x.double().numpy())
    tol = (cols / 32 + 160) * 2.0 ** -24 * a + HALF[out] * np.abs(ref) + 2.0 ** -25
    off = np.abs(y.double().cpu().numpy() - ref)
    assert y.dtype == out and np.all(off <= tol), (float((off / tol).max()), np.unravel_index((off / tol).argmax(), off.shape))


SHAPES = [
    # rows, cols, group
    (16, 128, 128), (1, 128, 128), (17, 256, 128), (33, 1024, 256), (1024, 1024, 256), (100, 4096, 128),
    (40, 640, 640), (48, 896, 448), (24, 384, 384),                # whole rows, groups that are no power of two
    (8, 256, 512), (6, 96, 288), (64, 64, 4096),                   # groups of several rows
    (50, 512, 64), (31, 544, 32), (70, 96, 32), (65, 32, 32), (19, 960, 64), (20, 480, 96), (16, 160, 160),
    (9, 100, 50), (7, 66, 33), (4, 3, 3), (2, 1, 2), (3, 42, 7), (10, 130, 26),   # any shape
    (130, 28672, 128), (20, 8160, 32)]


@pytest.mark.parametrize("rows,cols,group", SHAPES)
@pytest.mark.parametrize("batch,dtype,out,zp", [(1, F16, F16, True), (1, BF16, F32, True), (5, F16, F32, False),
                                                (13, BF16, BF16, True)])
def test_shapes(rows, cols, group, batch, dtype, out, zp):
    packed, scales, z, x = make(rows, cols, group, batch, dtype, zp)
    y = lt.gemv_int4(*dev(packed, scales, z), (rows, cols), group, x.to(DEV), dtype=out)
    check(y, packed, scales, z, rows, cols, group, x, out)


@pytest.mark.parametrize("batch", [2, 3, 4, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("rows,cols,group,dtype", [(72, 1024, 128, F16), (37, 1248, 32, BF16)])
def test_batches(batch, rows, cols, group, dtype):
    packed, scales, z, x = make(rows, cols, group, batch, dtype)
    y = lt.gemv_int4(*dev(packed, scales, z), (rows, cols), group, x.to(DEV))
    check(y, packed, scales, z, rows, cols, group, x, dtype)


@pytest.mark.parametrize("rows,cols,group", [(40, 512, 128), (40, 512, 64), (33, 544, 32), (9, 100, 50), (24, 384, 384)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_one_hot_columns_exact(rows, cols, group, dtype):
    """x = 1 at one column: (q - zp) s, one product, no rounding in fp32."""
    packed, scales, z, _ = make(rows, cols, group, 1, dtype)
    x = torch.zeros(16, cols, dtype=dtype)
    js = np.random.default_rng(3).integers(0, cols, 16)
    js[:4] = (0, cols - 1, 1, cols // 2)
    x[torch.arange(16), torch.from_numpy(js)] = 1.0
    y = lt.gemv_int4(*dev(packed, scales, z), (rows, cols), group, x.to(DEV), dtype=F32)
    ref, _ = ops4.gemv(packed, scales.view(np.uint16), z, rows, cols, group, x.double().numpy())
    assert np.array_equal(y.double().cpu().numpy(), ref)


def test_extreme_zero_points_and_scales():
    rows, cols, group = 48, 512, 128
    packed, scales, _, x = make(rows, cols, group, 3, F16)
    n = rows * cols // group
    z = np.resize(np.array([-128, 127, 0, 15], np.int8), n)
    scales = np.resize(np.array([6e-8, 1e-5, 0.0, 2.0, -0.5], np.float16), n)
    y = lt.gemv_int4(*dev(packed, scales, z), (rows, cols), group, x.to(DEV), dtype=F32)
    check(y, packed, scales, z, rows, cols, group, x, F32)


@pytest.mark.parametrize("dtype,sizes", [(F16, (6e-8, 1e-4, 6e4)), (BF16, (1e-30, 1e-3, 1e25))])
def test_small_and_large_vectors(dtype, sizes):
    """Rows of very different size in one call: each keeps its own precision."""
    rows, cols, group = 32, 512, 128
    packed, scales, z, x = make(rows, cols, group, 3, F32)
    x = (x * torch.tensor(sizes)[:, None]).clamp(-6e4 if dtype == F16 else -1e30, 6e4 if dtype == F16 else 1e30).to(dtype)
    y = lt.gemv_int4(*dev(packed, scales, z), (rows, cols), group, x.to(DEV), dtype=F32)
    check(y, packed, scales, z, rows, cols, group, x, F32)


@pytest.mark.parametrize("cols,group", [(512, 128), (544, 32), (100, 50)])
def test_not_finite_rows_stay_their_own(cols, group):
    rows = 33
    packed, scales, z, x = make(rows, cols, group, 4, F16)
    x[1, 3], x[2, cols - 1] = float("inf"), float("nan")
    y = lt.gemv_int4(*dev(packed, scales, z), (rows, cols), group, x.to(DEV))
    ok = [0, 3]
    check(y[ok], packed, scales, z, rows, cols, group, x[ok], F16)
    assert torch.isnan(y[2]).all()
    ref, _ = ops4.gemv(packed, scales.view(np.uint16), z, rows, cols, group, np.eye(1, cols, 3))
    hit = torch.from_numpy(ref[0] != 0)
    assert not torch.isfinite(y[1].cpu()[hit]).any()


@pytest.mark.parametrize("cols,group", [(512, 128), (544, 32), (66, 33)])
def test_strides_and_alignment(cols, group):
    """x and y as slices of wider tensors, at 16-byte and at odd offsets."""
    rows, batch = 40, 3
    packed, scales, z, x = make(rows, cols, group, batch, F16)
    for off, pad in ((0, 64), (8, 8), (1, 3), (2, 62)):
        wide = torch.full((batch, off + cols + pad), float("nan"), dtype=F16, device=DEV)
        wide[:, off:off + cols] = x.to(DEV)
        ywide = torch.full((batch, rows + 5), 7.0, dtype=F32, device=DEV)
        lt.gemv_int4(*dev(packed, scales, z), (rows, cols), group, wide[:, off:off + cols], y=ywide[:, 1:1 + rows])
        check(ywide[:, 1:1 + rows], packed, scales, z, rows, cols, group, x, F32)
        assert torch.all(ywide[:, 0] == 7.0) and torch.all(ywide[:, 1 + rows:] == 7.0)
    # codes that start off a 16-byte boundary
    raw = torch.zeros(packed.size + 4, dtype=torch.uint8, device=DEV)
    raw[4:] = torch.from_numpy(packed).to(DEV)
    y = lt.gemv_int4(raw[4:], *dev(packed, scales, z)[1:], (rows, cols), group, x.to(DEV), dtype=F32)
    check(y, packed, scales, z, rows, cols, group, x, F32)


def test_vector_form_same_bits_twice_and_side_stream():
    rows, cols, group = 512, 4096, 128
    packed, scales, z, x = make(rows, cols, group, 1, BF16)
    d, xd = dev(packed, scales, z), x.to(DEV)
    a = lt.gemv_int4(*d, (rows, cols), group, xd[0])
    assert a.shape == (rows,)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = torch.empty_like(a)
    lt.gemv_int4(*d, (rows, cols), group, xd[0], y=b, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b)
    check(a[None], packed, scales, z, rows, cols, group, x, BF16)


def test_agrees_with_dequant_and_product():
    """The weight that dequant_int4 writes, rounded to fp16 once more, gives the same product within that rounding."""
    rows, cols, group = 256, 2048, 128
    packed, scales, z, x = make(rows, cols, group, 2, F16)
    d, xd = dev(packed, scales, z), x.to(DEV)
    w = lt.dequant_int4(*d, (rows, cols), group).double()
    y = lt.gemv_int4(*d, (rows, cols), group, xd, dtype=F32).double()
    ref = xd.double() @ w.t()
    assert torch.all((y - ref).abs() <= (2.0 ** -11 + 224 * 2.0 ** -24) * (xd.double().abs() @ (w.abs() + 32 * 0.05).t()))
