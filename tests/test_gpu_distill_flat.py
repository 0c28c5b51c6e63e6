"""The loss of flat distributions with a remainder: a few entries that hold little of
either distribution, where the loss (1e-4 and less) is what is left of terms a
hundred times as large.

Tolerance. u = 2^-24. The loss is a function of the entries' log p and log q and of
what the exponentials and sums make of them:
  L = sum p (log p - log q) + (1 - P) (log(1 - P) - log(1 - Q)),  P = sum p, Q = sum q.
An exponential is 4 u relative, a sum over at most 16 entries 8 u, log(1 - P) 4 u of
itself (about P): together under 32 u (P + Q) with what the products add. An error
delta of a log p or a log q moves the entry's term and the remainder's, by
  p (log p - log q - log((1 - P) / (1 - Q))) delta  and  (q (1 - P) / (1 - Q) - p) delta.
log q is off by u for each of its parts (the exponent, under 32; the log of the sum,
under 16) and by the sum's own relative error (3 u |x| of an exponent, |x| <= 32, and
tree sums, 100 u), log p by 16 u: delta under 256 u."""
import numpy as np
import pytest
import torch

import quantized_sgd_amd as q

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q.lib()


# vocabularies of rows in registers, of one workgroup a row from memory, of rows in segments
@pytest.mark.parametrize("rows,vocab", [(5, 15296), (3, 101), (600, 70001), (2, 200003)])
@pytest.mark.parametrize("k", [1, 9, 16])
@pytest.mark.parametrize("tau", [4.0, 16.0])
def test_loss_of_flat_rows(rows, vocab, k, tau):
    g = torch.Generator().manual_seed(vocab + k)
    z = torch.randn(rows, vocab, generator=g) * 2.5
    zt = z * 0.8 + torch.randn(rows, vocab, generator=g) * 1.5
    t, idx = zt.topk(k, dim=1)
    lse = torch.logsumexp(zt.double() / tau, 1).float()
    loss, _ = q.distill_topk(z.cuda(), idx.cuda(), t.cuda(), tau=tau, teacher_lse=lse.cuda())
    step, _ = q.distill_topk_step(z.cuda(), idx.cuda(), t.cuda(), tau=tau, teacher_lse=lse.cuda())

    z64, lp = z.double() / tau, t.double() / tau - lse.double()[:, None]
    lq = z64.gather(1, idx) - torch.logsumexp(z64, 1, keepdim=True)
    p, s = lp.exp(), lq.exp()
    P, Q = p.sum(1), s.sum(1)
    rest = torch.log1p(-P) - torch.log1p(-Q)
    want = (p * (lp - lq)).sum(1) + (1 - P) * rest
    moved = (p * (lp - lq - rest[:, None])).abs().sum(1) + (s * ((1 - P) / (1 - Q))[:, None] - p).abs().sum(1)
    room = (32 * U * (P + Q) + 256 * U * moved).numpy()
    assert (P + Q < 1).all()
    assert (np.abs(loss.cpu().double().numpy() - want.numpy()) <= room).all()
    assert (np.abs(step.cpu().double().numpy() - want.numpy()) <= room).all()
