"""Distillation loss and gradient against the definition in 64 bits, and the
gradient against differences.

Tolerances. u = 2^-24. A probability q_j is exp2 of a rounded argument over a
rounded sum: the difference z - m and its product with log2(e) / tau leave an
absolute error of at most 3 u |x| in the exponent x = (z_j - m) / tau (natural
units, about 2^-22 |x|), the hardware's exp2 2 u, the sum of n terms in a tree of
per-thread runs (n / 512 + 20 additions, n <= 2^18) at most 600 u. So q_j is
relative 2^-13.5 off in the worst case that this test can reach and usually under
2^-20; with |x| <= 60 the bound below is
  |dq| <= 2^-13 q + 2^-24 (absolute: what exp2 leaves below its smallest normal).
p_i is a softmax over at most 1024 entries (under 2^-19 relative), and 2^-24 |t|
more with teacher_lse, where the remainder inherits the sum's error in absolute
terms. The loss adds |p| (|log p| + |log q|) times those. A gradient is then
rounded once to its type (2^-9 in bfloat16, 2^-12 in half precision, plus its
smallest subnormal)."""
import numpy as np
import pytest
import torch

import quantized_sgd_amd as q
from tests import plain_distill as plain

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -149), torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


def case(rows, vocab, k, dtype, seed, pad=0, offset=0, tail=False, tau=1.0, itype=torch.int32, ttype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 3
    zt = z * 0.7 + torch.randn(rows, vocab, generator=g)
    t, idx = zt.topk(min(k, vocab), dim=1)
    lse = torch.logsumexp(zt.double() / tau, 1).float().cuda() if tail else None
    flat = torch.zeros(rows * (vocab + pad) + offset).to(dtype).cuda()
    zz = flat[offset:].view(rows, vocab + pad)[:, :vocab]
    zz.copy_(z)
    weight = torch.rand(rows, generator=g) + 0.5
    return zz, idx.to(itype).cuda(), t.to(ttype).cuda(), lse, weight.cuda()


def close(got, want, dtype, scale):
    """|got - want| within the bound of the module's text; `scale` >= |want| is what
    the error goes by (sum of magnitudes that the value is made of)."""
    got, want = got.detach().cpu().double().numpy(), np.asarray(want)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    rel, tiny = ROUND[dtype]
    room = 2.0 ** -13 * scale + rel * np.abs(want) + tiny + 2.0 ** -24 * np.max(scale, axis=-1, keepdims=True)
    off = np.abs(got - want)
    assert (off[fine] <= np.broadcast_to(room, off.shape)[fine]).all(), float((off - room)[fine].max())


def check(z, idx, t, lse, weight, tau, out=None):
    zh, ih, th = z.detach().cpu().double().numpy(), idx.cpu().numpy(), t.cpu().double().numpy()
    lh = None if lse is None else lse.cpu().double().numpy()
    gh = None if weight is None else weight.cpu().double().numpy()
    loss, dz = plain.rows(zh, ih, th, tau, lh, gh)
    kept = z.clone()
    step_loss, step_dz = q.distill_topk_step(z, idx, t, weight, tau=tau, teacher_lse=lse, out=out)
    assert torch.equal(z.view(torch.uint8), kept.view(torch.uint8)) if z.is_contiguous() else True
    got, stats = q.distill_topk(z, idx, t, tau=tau, teacher_lse=lse)
    got_dz = q.distill_topk_backward(z, idx, t, stats, weight, tau=tau, teacher_lse=lse)
    # magnitudes: the loss is made of terms p (log p - log q) of up to 1 x 60 each and cancels at worst to 0
    near = np.where(np.isfinite(loss), 1.0 + np.abs(loss), 1.0)
    close(got, loss, torch.float32, near)
    close(step_loss, loss, torch.float32, near)
    w = np.ones(len(zh)) if gh is None else np.abs(gh)
    scale = np.where(np.isfinite(dz), np.abs(dz), 0) + (w / tau)[:, None] * _mass(zh, ih, th, tau, lh)
    close(got_dz, dz, z.dtype, scale)
    close(step_dz, dz, z.dtype, scale)
    return step_loss, step_dz


def _mass(z, idx, t, tau, lse):
    """q_j + p_j (and the remainder's share): what a gradient's difference is taken of."""
    out = np.zeros(z.shape)
    for i in range(len(z)):
        _, d = plain.row(z[i], idx[i], t[i], tau, None if lse is None else lse[i])
        x = z[i] / tau
        with np.errstate(all="ignore"):
            e = np.nan_to_num(np.exp(x - np.nanmax(np.where(np.isposinf(x), -np.inf, x))))
        s = e.sum()
        out[i] = (2 * e / s if s > 0 else 0) + np.nan_to_num(np.abs(d))
    return out


SHAPES = [(1, 1, 1), (1, 2, 1), (2, 7, 3), (3, 8, 8), (5, 63, 4), (4, 513, 16), (3, 4097, 32), (2, 8192, 64), (300, 1000, 5), (7, 16385, 20),
          (1, 100003, 50), (260, 4100, 8), (2, 262145, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,k", SHAPES)
def test_loss_and_gradient(rows, vocab, k, dtype):
    for pad, offset, tail, tau, itype, ttype in [(0, 0, False, 1.0, torch.int32, torch.float32),
                                                 (3, 1, True, 2.0, torch.int64, torch.bfloat16)]:
        print("distill", rows, vocab, k, dtype, pad, tail, flush=True)
        z, idx, t, lse, w = case(rows, vocab, k, dtype, rows + vocab, pad, offset, tail, tau, itype, ttype)
        check(z, idx, t, lse, w, tau)
        if rows < 10 and vocab < 5000:
            check(z, idx, t, lse, None, tau)


@pytest.mark.parametrize("k", [1, 64, 511, 512, 513, 1024])
@pytest.mark.parametrize("tail", [False, True])
def test_many_entries(k, tail):
    z, idx, t, lse, w = case(4, 1500, k, torch.float32, k, tail=tail)
    check(z, idx, t, lse, w, 1.0)


@pytest.mark.parametrize("rows,vocab", [(6, 600), (6, 40000)])
@pytest.mark.parametrize("tail", [False, True])
def test_rows_that_masks_leave_little_of(rows, vocab, tail):
    z, idx, t, lse, w = case(rows, vocab, 12, torch.float32, 9, tail=tail)
    idx[0] = -1                        # no entries
    idx[1, 3:] = vocab                 # past the vocabulary: no entry
    idx[1, 4] = 2 ** 31 - 1
    w[2] = 0.0                         # weighs nothing
    z[3, 100:] = -torch.inf            # vocabulary that the student lacks
    idx[3] = torch.arange(12, device="cuda", dtype=idx.dtype)
    lowest = torch.finfo(torch.float32).min
    z[4, 50:] = lowest                 # masked with the type's lowest value instead
    idx[4] = torch.arange(12, device="cuda", dtype=idx.dtype)
    t[5, 6:] = -torch.inf              # entries that the teacher gives nothing
    check(z, idx, t, lse, w, 1.0)
    # no remainder at all: everything outside the entries is masked
    z[3, 12:] = -torch.inf
    check(z[3:4], idx[3:4], t[3:4], None if lse is None else lse[3:4], w[3:4], 1.0)


@pytest.mark.parametrize("tail", [False, True])
def test_infinite_and_not_a_number(tail):
    z, idx, t, lse, w = case(6, 700, 5, torch.float32, 3, tail=tail)
    z[0] = -torch.inf                  # a student without any vocabulary
    z[1, 650] = torch.nan
    z[2, 650] = torch.inf
    z[3, idx[3, 0].long()] = -torch.inf   # an entry that the student gives nothing
    z[4, idx[4, 0].long()] = torch.nan
    idx[5] = -1
    z[5] = torch.nan                   # a row without entries: zeros whatever its logits
    check(z, idx, t, lse, w, 1.0)
    w[:] = 0
    _, dz = q.distill_topk_step(z, idx, t, w, teacher_lse=lse)
    assert torch.equal(dz, torch.zeros_like(dz))


def test_large_logits():
    # a shift of all logits changes nothing: 1e4 + z in fp32 keeps z to 2^-10
    z, idx, t, lse, w = case(4, 900, 6, torch.float32, 8, tail=True)
    z.copy_((z * 64).round() / 64)
    a, da = q.distill_topk_step(z, idx, t, w, teacher_lse=lse)
    b, db = q.distill_topk_step(z + 8192.0, idx, t, w, teacher_lse=lse)
    assert torch.equal(a, b) and torch.equal(da, db)


def test_a_student_sure_of_the_entries():
    # the remainder is e-30 of the student's mass: it has to come from its own sum
    z, idx, t, lse, w = case(3, 2000, 4, torch.float32, 8, tail=True)
    for i in range(3):
        z[i, idx[i].long()] += 70.0
    check(z, idx, t, lse, w, 1.0)


@pytest.mark.parametrize("rows,vocab", [(5, 3001), (3, 70001), (300, 520)])
def test_in_place(rows, vocab):
    z, idx, t, lse, w = case(rows, vocab, 9, torch.bfloat16, 4, pad=3, tail=True)
    loss, dz = q.distill_topk_step(z, idx, t, w, teacher_lse=lse)
    _, stats = q.distill_topk(z, idx, t, teacher_lse=lse)
    a, b = z.clone(), z.clone()
    loss2, same = q.distill_topk_step(a, idx, t, w, teacher_lse=lse, out=a)
    assert same is a and torch.equal(a, dz) and torch.equal(loss, loss2)
    q.distill_topk_backward(b, idx, t, stats, w, teacher_lse=lse, out=b)
    assert torch.equal(b, q.distill_topk_backward(z, idx, t, stats, w, teacher_lse=lse))


def test_writes_nothing_else():
    for dtype, vocab in [(torch.bfloat16, 1003), (torch.float32, 20001), (torch.float16, 5)]:
        z, idx, t, lse, w = case(5, vocab, 3, dtype, 2)
        buf = torch.full((5 * (vocab + 3) + 128,), 9.0, dtype=dtype, device="cuda")
        out = buf[64:64 + 5 * (vocab + 3)].view(5, vocab + 3)[:, :vocab]
        q.distill_topk_step(z, idx, t, w, out=out)
        assert torch.equal(out, q.distill_topk_step(z, idx, t, w)[1])
        out.fill_(9.0)
        assert bool((buf == 9.0).all())


def test_nothing():
    z = torch.empty(0, 10, device="cuda")
    idx, t = torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, 3, device="cuda")
    loss, dz = q.distill_topk_step(z, idx, t)
    assert loss.shape == (0,) and dz.shape == (0, 10)
    z = torch.randn(4, 10, device="cuda")
    idx, t = torch.empty(4, 0, dtype=torch.int32, device="cuda"), torch.empty(4, 0, device="cuda")
    loss, dz = q.distill_topk_step(z, idx, t)
    assert torch.equal(loss, torch.zeros_like(loss)) and torch.equal(dz, torch.zeros_like(z))
    z = torch.empty(4, 0, device="cuda")
    loss, dz = q.distill_topk_step(z, torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda"))
    assert torch.equal(loss.cpu(), torch.zeros(4)) and dz.shape == (4, 0)


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(tail):
    """Central differences of the 64-bit loss: with steps of 2^-7 their own error is
    below h^2 / 6 times a third derivative of at most 1 (1.1e-5)."""
    z, idx, t, lse, _ = case(3, 40, 5, torch.float32, 6, tail=tail, tau=2.0)
    _, dz = q.distill_topk_step(z, idx, t, tau=2.0, teacher_lse=lse)
    zh, ih, th = z.cpu().double().numpy(), idx.cpu().numpy(), t.cpu().double().numpy()
    lh = [None] * 3 if lse is None else lse.cpu().double().numpy()
    h = 2.0 ** -7
    for i in range(3):
        for j in range(40):
            up, dn = zh[i].copy(), zh[i].copy()
            up[j] += h
            dn[j] -= h
            diff = (plain.row(up, ih[i], th[i], 2.0, lh[i])[0] - plain.row(dn, ih[i], th[i], 2.0, lh[i])[0]) / (2 * h)
            assert abs(diff - float(dz[i, j])) < 2e-5


def test_another_stream_and_repeats():
    z, idx, t, lse, w = case(5, 50001, 20, torch.bfloat16, 7, tail=True)
    loss, dz = q.distill_topk_step(z, idx, t, w, teacher_lse=lse)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    loss2, dz2 = q.distill_topk_step(z, idx, t, w, teacher_lse=lse, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(dz, dz2)


def test_graph_replays():
    z, idx, t, lse, w = case(4, 30000, 8, torch.float16, 1, tail=True)

    def step():
        loss, stats = q.distill_topk(z, idx, t, teacher_lse=lse)
        return loss, q.distill_topk_backward(z, idx, t, stats, w, teacher_lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (2, 3, 4):
        z.copy_(case(4, 30000, 8, torch.float16, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_refusals():
    z, idx, t, lse, w = case(4, 50, 3, torch.float32, 1, tail=True)
    bad = [lambda: q.distill_topk(z.double(), idx, t), lambda: q.distill_topk(z.cpu(), idx, t),
           lambda: q.distill_topk(z, idx[:3], t), lambda: q.distill_topk(z, idx, t[:, :2]),
           lambda: q.distill_topk(z, idx.float(), t), lambda: q.distill_topk(z, idx, t.int()),
           lambda: q.distill_topk(z, idx, t, tau=0.0), lambda: q.distill_topk(z, idx, t, tau=-1.0),
           lambda: q.distill_topk(z, idx, t, tau=float("nan")), lambda: q.distill_topk(z, idx, t, tau=float("inf")),
           lambda: q.distill_topk(z, idx, t, teacher_lse=lse[:2]), lambda: q.distill_topk(z[0], idx, t),
           lambda: q.distill_topk(z, idx.cpu(), t),
           lambda: q.distill_topk(z, idx.repeat(1, 400), t.repeat(1, 400)),
           lambda: q.distill_topk_step(z, idx, t, w[:3]), lambda: q.distill_topk_step(z, idx, t, w.double()),
           lambda: q.distill_topk_step(z, idx, t, w, out=z.half()),
           lambda: q.distill_topk_step(z, idx, t, w, out=torch.empty(4, 51, device="cuda")),
           lambda: q.distill_topk_step(z, idx, t, w, out=z.view(-1)[:200].view(50, 4).t()),
           lambda: q.distill_topk_backward(z, idx, t, torch.zeros(4, 3, device="cuda")),
           lambda: q.distill_topk_backward(z, idx, t, torch.zeros(3, 4, device="cuda"))]
    for i, f in enumerate(bad):
        print("refusal", i, flush=True)
        with pytest.raises(ValueError):
            f()
