"""Offsets past 32 bits: row strides so large that the later rows of a matrix start
beyond 2^31 elements (and 2^32 bytes). The same rows in a compact matrix give the
expected results bit for bit."""
import pytest
import torch

import quantized_sgd_amd as q

pytestmark = pytest.mark.gpu
STRIDE = (1 << 30) + 24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GB of device memory")
    q.lib()


def far(rows, cols, dtype):
    """A matrix whose rows lie STRIDE elements apart."""
    return torch.empty((rows - 1) * STRIDE + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (STRIDE, 1))


def test_quantize_far_rows():
    x = torch.randn(5, 700, device="cuda").bfloat16()
    wide = far(5, 700, torch.bfloat16)
    wide.copy_(x)
    for transpose in (False, True):
        a, sa = q.int8_quantize(x, transpose=transpose)
        out = far(*a.shape, torch.int8) if not transpose else None
        b, sb = q.int8_quantize(wide, transpose=transpose, out=out)
        assert torch.equal(a, b) and torch.equal(sa, sb)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [4, 40])
def test_product_of_far_rows(m):
    # m rows of a compact; b and y far apart (b is copied to aligned rows for the tiles)
    k, n = 128, 5
    a = torch.randint(-127, 128, (m, k), dtype=torch.int8, device="cuda")
    b = torch.randint(-127, 128, (n, k), dtype=torch.int8, device="cuda")
    sa, sb = torch.rand(m, device="cuda"), torch.rand(n, device="cuda")
    wide = far(n, k, torch.int8)
    wide.copy_(b)
    assert torch.equal(q.int8_matmul(a, sa, b, sb), q.int8_matmul(a, sa, wide, sb))
    y = far(4, n, torch.float32)
    q.int8_matmul(a[:4], sa[:4], b, sb, out=y)
    assert torch.equal(y, q.int8_matmul(a[:4], sa[:4], b, sb, dtype=torch.float32))
    y = far(2, n, torch.float32)
    torch.cuda.empty_cache()


def test_tile_rows_far_apart():
    # y of the tiles with rows past 2^31 elements
    m, k, n = 33, 64, 70
    stride = (1 << 26) + 16
    a = torch.randint(-127, 128, (m, k), dtype=torch.int8, device="cuda")
    b = torch.randint(-127, 128, (n, k), dtype=torch.int8, device="cuda")
    sa = torch.rand(m, device="cuda")
    y = torch.empty((m - 1) * stride + n, dtype=torch.float32, device="cuda").as_strided((m, n), (stride, 1))
    q.int8_matmul(a, sa, b, out=y)
    assert torch.equal(y, q.int8_matmul(a, sa, b, dtype=torch.float32))
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("vocab", [1000, 200_000])
def test_distill_far_rows(vocab):
    z = torch.randn(4, vocab, device="cuda").bfloat16()
    t, idx = z.float().topk(9, dim=1)
    lse = torch.logsumexp(z.float(), 1)
    g = torch.rand(4, device="cuda")
    wide, out = far(4, vocab, torch.bfloat16), far(4, vocab, torch.bfloat16)
    wide.copy_(z)
    loss, dz = q.distill_topk_step(z, idx, t, g, teacher_lse=lse)
    loss2, dz2 = q.distill_topk_step(wide, idx, t, g, teacher_lse=lse, out=out)
    assert torch.equal(loss, loss2) and torch.equal(dz, dz2)
    _, stats = q.distill_topk(wide, idx, t, teacher_lse=lse)
    assert torch.equal(q.distill_topk_backward(wide, idx, t, stats, g, teacher_lse=lse, out=out), dz)
    del wide, out
    torch.cuda.empty_cache()
