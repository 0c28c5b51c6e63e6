"""The 8-bit linear layer against its definition on the CPU. Every step is a
single IEEE rounding of an exactly known value (integer sums are exact), so the
results must be equal, not near; only the comparison of the gradient with the
derivative in reals has a tolerance, which follows from the 8-bit rounding of gy
(half a level for each term)."""
import numpy as np
import pytest
import torch

import quantized_sgd_amd as q
from tests import plain_int8 as plain

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def values(rows, cols, dtype, seed, pad=0, offset=0, scale=1.0):
    """[rows, cols] on the device, as a view with `pad` more columns and an odd
    start where asked."""
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(rows * (cols + pad) + offset, generator=g) * scale
    return flat.to(dtype).cuda()[offset:].view(rows, cols + pad)[:, :cols]


def levels(rows, cols, seed, pad=0, offset=0, low=-127):
    g = torch.Generator().manual_seed(seed)
    flat = torch.randint(low, 128, (rows * (cols + pad) + offset,), generator=g, dtype=torch.int8)
    return flat.cuda()[offset:].view(rows, cols + pad)[:, :cols]


def scales(n, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(n, generator=g) + 0.25).cuda()


def guarded(rows, cols, pad, dtype, fill):
    """An output view inside a buffer whose other elements must stay `fill`."""
    buf = torch.full((64 + rows * (cols + pad) + 64,), fill, dtype=dtype, device="cuda")
    view = buf[64:64 + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return buf, view


def untouched(buf, view, fill):
    view.fill_(fill)
    return bool((buf == fill).all())


# ---- quantizer ----

SHAPES = [(1, 1), (1, 7), (3, 8), (2, 64), (5, 511), (4, 512), (7, 1000), (3, 1024), (2, 2047), (130, 33), (3, 4096), (2, 5003),
          (2, 8192), (1, 16383), (2, 16385), (1, 40001), (129, 65), (256, 128), (1021, 77)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_rows(rows, cols, dtype):
    for pad, offset, folded in [(0, 0, False), (5, 1, True)]:
        print("quantize", rows, cols, dtype, pad, offset, folded, flush=True)
        x = values(rows, cols, dtype, rows + cols, pad, offset)
        fold = scales(cols, 3) if folded else None
        buf, out = guarded(rows, cols, pad, torch.int8, 99)
        got, s = q.int8_quantize(x, fold=fold, out=out)
        want, ws = plain.quantize_rows(plain.to32(x), None if fold is None else plain.to32(fold))
        assert np.array_equal(s.cpu().numpy(), ws)
        assert np.array_equal(got.cpu().numpy(), want)
        assert untouched(buf, out, 99)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_columns(rows, cols, dtype):
    for pad, offset, folded in [(0, 0, False), (3, 1, True)]:
        print("quantize columns", rows, cols, dtype, pad, offset, folded, flush=True)
        x = values(rows, cols, dtype, rows * 3 + cols, pad, offset)
        fold = scales(rows, 5) if folded else None
        buf, out = guarded(cols, rows, pad, torch.int8, 99)
        got, s = q.int8_quantize(x, fold=fold, transpose=True, out=out)
        want, ws = plain.quantize_columns(plain.to32(x), None if fold is None else plain.to32(fold))
        assert np.array_equal(s.cpu().numpy(), ws)
        assert np.array_equal(got.cpu().numpy(), want)
        assert untouched(buf, out, 99)


def _hard_rows():
    """Rows where rounding or range can go wrong."""
    sub = np.float32(2.0) ** -149
    tie = np.zeros(300, np.float32)
    tie[0] = 127.0                      # scale 1: halves are exact ties
    tie[1:255] = np.arange(-127, 127) + 0.5
    near = np.zeros(300, np.float32)
    near[0] = 127.0
    near[1:255] = np.nextafter((np.arange(-127, 127) + 0.5).astype(np.float32), np.float32(1e9))
    rows = [np.zeros(300, np.float32), tie, near, np.nextafter(near, np.float32(-1e9)), np.full(300, sub),
            np.linspace(-190, 190, 300).astype(np.float32).round() * sub,      # a subnormal scale that is too small
            np.linspace(-3e38, 3e38, 300).astype(np.float32), np.linspace(-1e-38, 1e-38, 300).astype(np.float32),
            np.linspace(-1, 1, 300).astype(np.float32) / 3]
    for bad in (np.inf, -np.inf, np.nan):
        r = np.linspace(-1, 1, 300).astype(np.float32)
        r[17] = bad
        rows.append(r)
    minus = np.full(300, -0.0, np.float32)
    rows.append(minus)
    return np.stack(rows)


def test_quantize_extremes():
    x = _hard_rows()
    want, ws = plain.quantize_rows(x)
    for transpose in (False, True):
        t = torch.from_numpy(np.ascontiguousarray(x.T if transpose else x)).cuda()
        got, s = q.int8_quantize(t, transpose=transpose)
        assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
        assert np.array_equal(got.cpu().numpy(), want)


def test_quantize_nothing():
    for r, c in [(0, 5), (5, 0), (0, 0)]:
        x = torch.empty(r, c, device="cuda")
        levels_, s = q.int8_quantize(x)
        assert levels_.shape == (r, c) and torch.equal(s.cpu(), torch.zeros(r))
        levels_, s = q.int8_quantize(x, transpose=True)
        assert levels_.shape == (c, r) and torch.equal(s.cpu(), torch.zeros(c))


# ---- product ----

PRODUCTS = [(1, 1, 1), (1, 1, 16), (1, 5, 17), (2, 16, 64), (3, 33, 65), (1, 128, 4096), (16, 100, 1040), (17, 64, 48), (32, 200, 333),
            (33, 31, 64), (33, 65, 80), (64, 64, 64), (65, 63, 128), (100, 130, 15), (128, 128, 256), (129, 257, 272), (300, 200, 1000),
            (515, 1100, 208), (40, 40, 9000), (1024, 1300, 64), (2100, 3000, 144)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k, dtype):
    for pad, offset, extra in [(0, 0, False), (16, 0, True), (3, 5, True)]:
        print("product", m, n, k, dtype, pad, offset, flush=True)
        a, b = levels(m, k, m + k, pad, offset, -128), levels(n, k, n + k + 1, pad, offset, -128)
        sa, sb = scales(m, 1), scales(n, 2) if extra else None
        bias = scales(n, 3) - 0.5 if extra else None
        buf, out = guarded(m, n, pad, dtype, 7.0)
        y = q.int8_matmul(a, sa, b, sb, bias=bias, out=out)
        want = plain.product(a.cpu().numpy(), plain.to32(sa), b.cpu().numpy(), None if sb is None else plain.to32(sb),
                             None if bias is None else plain.to32(bias))
        assert plain.same(y, plain.cast(want, dtype))
        assert untouched(buf, out, 7.0)


def test_product_large_tiles():
    # enough tiles for the largest tile, ragged in every direction
    m, n, k = 3600, 4200, 336
    a, b, sa, sb = levels(m, k, 1), levels(n, k, 2), scales(m, 3), scales(n, 4)
    y = q.int8_matmul(a, sa, b, sb, dtype=torch.float32)
    assert plain.same(y, torch.from_numpy(plain.product(a.cpu().numpy(), plain.to32(sa), b.cpu().numpy(), plain.to32(sb))))


@pytest.mark.parametrize("m", [1, 40])
def test_product_sums_past_32_bits(m):
    # every product at its largest: the sum passes 2^31 and is still exact
    k = 150_016
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    b = torch.full((33, k), -128, dtype=torch.int8, device="cuda")
    b[1] = 127
    b[2, ::2] = 127
    y = q.int8_matmul(a, torch.ones(m, device="cuda"), b, dtype=torch.float32)
    want = plain.product(a.cpu().numpy(), np.ones(m), b.cpu().numpy())
    assert want.max() > 2.0 ** 31 and plain.same(y, torch.from_numpy(want))


def test_product_without_a_sum():
    sa, bias = scales(3, 1), scales(40, 2)
    for m in (3, 70):
        a, b = torch.empty(m, 0, dtype=torch.int8, device="cuda"), torch.empty(40, 0, dtype=torch.int8, device="cuda")
        y = q.int8_matmul(a, scales(m, 1), b, bias=bias, dtype=torch.float32)
        assert torch.equal(y, bias.expand(m, 40))
    assert q.int8_matmul(torch.empty(0, 8, dtype=torch.int8, device="cuda"), scales(0, 1), levels(4, 8, 1)).shape == (0, 4)
    assert q.int8_matmul(levels(3, 8, 1), sa, torch.empty(0, 8, dtype=torch.int8, device="cuda")).shape == (3, 0)


def test_product_special_scales():
    # infinite, zero and NaN scales go through the epilogue's products as they are
    a, b = levels(40, 64, 1), levels(50, 64, 2)
    sa, sb = scales(40, 3), scales(50, 4)
    sa[0], sa[1], sa[2], sb[3], sb[4] = np.inf, 0.0, np.nan, np.inf, 0.0
    y = q.int8_matmul(a, sa, b, sb, dtype=torch.float32)
    assert plain.same(y, torch.from_numpy(plain.product(a.cpu().numpy(), plain.to32(sa), b.cpu().numpy(), plain.to32(sb))))


# ---- layer and gradient ----

LAYERS = [(1, 1, 1), (1, 100, 64), (1, 256, 4096), (2, 33, 1000), (7, 64, 48), (16, 129, 515), (24, 301, 2048), (33, 70, 130),
          (100, 77, 153), (300, 260, 200), (1000, 777, 1537)]


def _layer(x, w, sw, bias):
    xq, sx = plain.quantize_rows(plain.to32(x))
    return xq, sx, plain.product(xq, sx, w.cpu().numpy(), plain.to32(sw), None if bias is None else plain.to32(bias))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", LAYERS)
def test_linear(m, n, k, dtype):
    for pad, offset in [(0, 0), (7, 3)]:
        print("linear", m, n, k, dtype, pad, offset, flush=True)
        x, w, sw = values(m, k, dtype, m + n, pad, offset), levels(n, k, k, pad, offset), scales(n, 2)
        bias = scales(n, 4) if offset else None
        xq, sx, want = _layer(x, w, sw, bias)
        y = q.int8_linear(x, w, sw, bias=bias)
        assert plain.same(y, plain.cast(want, dtype))
        y2, gq, gs = q.int8_linear(x, w, sw, bias=bias, keep=True)
        assert torch.equal(y, y2) and np.array_equal(gq.cpu().numpy(), xq) and np.array_equal(gs.cpu().numpy(), sx)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", LAYERS)
def test_linear_backward(m, n, k, dtype):
    print("backward", m, n, k, dtype, flush=True)
    x, w, sw = values(m, k, dtype, 5), levels(n, k, 6, 1), scales(n, 7)
    gy = values(m, n, dtype, 8, 3, 1, 0.01)
    _, xq, sx = q.int8_linear(x, w, sw, keep=True)
    gx, gw = q.int8_linear_backward(gy, xq, sx, w, sw)
    g32, xq_, w_ = plain.to32(gy), xq.cpu().numpy(), w.cpu().numpy()
    gq, sg = plain.quantize_rows(g32, plain.to32(sw))
    hq, sh = plain.quantize_columns(g32, plain.to32(sx))
    assert plain.same(gx, plain.cast(plain.product(gq, sg, w_.T), dtype))
    assert plain.same(gw, torch.from_numpy(plain.product(hq, sh, xq_.T)))
    # only one of the two
    gx1, none = q.int8_linear_backward(gy, xq, sx, w, sw, need_gw=False)
    assert none is None and torch.equal(gx1, gx)
    none, gw1 = q.int8_linear_backward(gy, xq, sx, w, sw, need_gx=False)
    assert none is None and torch.equal(gw1, gw)


@pytest.mark.parametrize("m,n,k", [(3, 5, 4), (20, 64, 48), (70, 33, 129)])
def test_gradient_against_differences(m, n, k):
    """L = sum gy y is linear in the real factors X = sx xq and W = sw w, so its
    differences are the derivative exactly (in 64 bits, steps of 1): they may be
    off from gx and gw by half a level of gy for each term, and by fp32 roundings
    (below 2^-21 of the sum of magnitudes: 7 roundings of 2^-24)."""
    x, w, sw, gy = values(m, k, torch.float32, 1), levels(n, k, 2), scales(n, 3), values(m, n, torch.float32, 4)
    _, xq, sx = q.int8_linear(x, w, sw, keep=True)
    gx, gw = (t.cpu().double().numpy() for t in q.int8_linear_backward(gy, xq, sx, w, sw))
    xr = xq.cpu().double().numpy() * sx.cpu().double().numpy()[:, None]
    wr = w.cpu().double().numpy() * sw.cpu().double().numpy()[:, None]
    g = gy.cpu().double().numpy()
    loss = lambda a, b: float((g * (a @ b.T)).sum())  # noqa: E731
    _, sg = plain.quantize_rows(plain.to32(gy), plain.to32(sw))
    _, sh = plain.quantize_columns(plain.to32(gy), plain.to32(sx))
    rng = np.random.default_rng(5)
    for _ in range(20):
        i, p, j = rng.integers(m), rng.integers(k), rng.integers(n)
        up, dn = xr.copy(), xr.copy()
        up[i, p] += 1.0
        dn[i, p] -= 1.0
        diff = (loss(up, wr) - loss(dn, wr)) / 2
        room = np.abs(w.cpu().double().numpy()[:, p]).sum() * sg[i] / 2 + 2.0 ** -21 * np.abs(g[i] @ np.abs(wr)).max() + 1e-9
        assert abs(diff - gx[i, p]) <= room
        up, dn = wr.copy(), wr.copy()
        up[j, p] += 1.0
        dn[j, p] -= 1.0
        diff = (loss(xr, up) - loss(xr, dn)) / 2
        room = np.abs(xq.cpu().double().numpy()[:, p]).sum() * sh[j] / 2 + 2.0 ** -21 * (np.abs(g[:, j]) @ np.abs(xr)).max() + 1e-9
        assert abs(diff - gw[j, p]) <= room


def test_nothing_to_multiply():
    w, sw = levels(5, 8, 1), scales(5, 1)
    y, xq, sx = q.int8_linear(torch.empty(0, 8, device="cuda"), w, sw, keep=True)
    assert y.shape == (0, 5) and xq.shape == (0, 8) and sx.shape == (0,)
    gx, gw = q.int8_linear_backward(torch.empty(0, 5, device="cuda"), xq, sx, w, sw)
    assert gx.shape == (0, 8) and torch.equal(gw.cpu(), torch.zeros(5, 8))
    x = torch.randn(3, 8, device="cuda")
    w0, sw0 = torch.empty(0, 8, dtype=torch.int8, device="cuda"), scales(0, 1)
    y, xq, sx = q.int8_linear(x, w0, sw0, keep=True)
    assert y.shape == (3, 0)
    gx, gw = q.int8_linear_backward(torch.empty(3, 0, device="cuda"), xq, sx, w0, sw0)
    assert torch.equal(gx.cpu(), torch.zeros(3, 8)) and gw.shape == (0, 8)
    y, xq, sx = q.int8_linear(torch.empty(3, 0, device="cuda"), torch.empty(5, 0, dtype=torch.int8, device="cuda"), sw,
                              bias=sw, keep=True)
    assert torch.equal(y, sw.expand(3, 5)) and xq.shape == (3, 0)


def test_poisoned_rows_stay_apart():
    # an infinity or NaN in one token or channel shows in that one's results only
    x, w, sw = values(40, 96, torch.float32, 1), levels(50, 96, 2), scales(50, 3)
    clean = q.int8_linear(x, w, sw)
    x[5, 7], x[9, 0] = np.inf, np.nan
    y = q.int8_linear(x, w, sw)
    assert y[5].isnan().all() and y[9].isnan().all()
    keep = [i for i in range(40) if i not in (5, 9)]
    assert torch.equal(y[keep], clean[keep])


def test_another_stream():
    x, w, sw = values(100, 256, torch.bfloat16, 1), levels(300, 256, 2), scales(300, 3)
    y, xq, sx = q.int8_linear(x, w, sw, keep=True)
    gy = values(100, 300, torch.bfloat16, 4)
    gx, gw = q.int8_linear_backward(gy, xq, sx, w, sw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, xq2, sx2 = q.int8_linear(x, w, sw, keep=True, stream=side)
    gx2, gw2 = q.int8_linear_backward(gy, xq2, sx2, w, sw, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(gx, gx2) and torch.equal(gw, gw2)


def test_graph_replays():
    x, w, sw = values(24, 512, torch.float16, 1), levels(300, 512, 2), scales(300, 3)
    gy = values(24, 300, torch.float16, 5)

    def step():
        y, xq, sx = q.int8_linear(x, w, sw, keep=True)
        return (y, *q.int8_linear_backward(gy, xq, sx, w, sw))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (11, 12, 13):
        x.copy_(values(24, 512, torch.float16, seed))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


# ---- refusals ----

def test_refusals():
    a, b, sa = levels(4, 8, 1), levels(6, 8, 2), scales(4, 3)
    x, sw = values(4, 8, torch.float32, 1), scales(6, 4)
    bad = [lambda: q.int8_matmul(a.float(), sa, b), lambda: q.int8_matmul(a, sa, levels(6, 9, 1)),
           lambda: q.int8_matmul(a, sa[:3], b), lambda: q.int8_matmul(a, sa.double(), b), lambda: q.int8_matmul(a, None, b),
           lambda: q.int8_matmul(a, sa, b, bias=sa), lambda: q.int8_matmul(a.cpu(), sa, b),
           lambda: q.int8_matmul(a, sa, b.cpu()), lambda: q.int8_matmul(levels(8, 4, 1).t(), sa, b),
           lambda: q.int8_matmul(a, sa, b, out=torch.empty(4, 7, device="cuda")),
           lambda: q.int8_matmul(a, sa, b, out=torch.empty(4, 6, dtype=torch.float64, device="cuda")),
           lambda: q.int8_matmul(a, sa, b, out=torch.empty(6, 4, device="cuda").t()),
           lambda: q.int8_matmul(a[0], sa, b), lambda: q.int8_quantize(x.double()), lambda: q.int8_quantize(x.cpu()),
           lambda: q.int8_quantize(x, fold=sa), lambda: q.int8_quantize(x, out=torch.empty(4, 9, dtype=torch.int8, device="cuda")),
           lambda: q.int8_quantize(x.t()), lambda: q.int8_quantize(x[:1].expand(4, 8)),
           lambda: q.int8_linear(x, b, scales(5, 1)), lambda: q.int8_linear(x, b.half(), sw),
           lambda: q.int8_linear(x, b, sw, out=torch.empty(4, 6, dtype=torch.float16, device="cuda")),
           lambda: q.int8_linear_backward(values(4, 6, torch.float32, 1), a, sa, b, sa),
           lambda: q.int8_linear_backward(values(3, 6, torch.float32, 1), a, sa, b, sw)]
    for i, f in enumerate(bad):
        print("refusal", i, flush=True)
        with pytest.raises(ValueError):
            f()
