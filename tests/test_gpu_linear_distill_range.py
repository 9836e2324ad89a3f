"""The loss of linear_distillation where the logits over the temperature are large:
low temperatures, and logits that all tokens' words have a common offset in.  The
divergence does not depend on the offset, and its terms are differences from the
row's largest logit.

Logits here are whole multiples of 2^-6 below 2^12, which fp32 sums hold exactly in
any order.  Tolerances, derived beforehand, u = 2^-24, d = (z - max z) / t:

* the sum of exponentials: an argument off by 3 u |d| (factor, product, difference),
  an exponential of 2^-22, and on the way to the row's sum at most 24 steps that add
  (u each) or rescale (2^-22 each, 8 of them), so log sum off by 2^-18 and 6 u of the
  mean of |d| under p;
* a term q (log q - (d - log sum)): q off by (2 |a| + 10) u of itself, where a is the
  exponential's argument, met times |log q - log p| + 1; the term's own roundings, 4 u of
  |log q| + |d| + log sum.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


def eighths(shape, g):
    return torch.randint(-8, 9, shape, generator=g) / 8


# the entries' logits taken from w again; picked out of tiles whose rows are words;
# and out of tiles whose rows are tokens
@pytest.mark.parametrize("rows,k", [(24, 32), (100, 64), (300, 40)])
@pytest.mark.parametrize("t,offset", [(1.0, 0), (1.0, 2048), (2.5, 2048), (0.05, 0), (0.05, 256),
                                      (2.0 ** -10, 64), (2.0 ** -20, 0)])
def test_loss(bo, rows, k, t, offset):
    g = torch.Generator().manual_seed(rows + offset)
    dim, vocab = 64, 1000
    x, w = eighths((rows, dim), g), eighths((vocab, dim), g)
    x[:, 0], w[:, 0] = offset / 64, 64 if offset else 0
    x, w = x.half().cuda(), w.half().cuda()
    t = float(torch.tensor(t).float())
    z = x.double() @ w.double().T
    top = z.amax(1, keepdim=True)
    # a teacher near the student, of the words that count
    zk, ids = torch.topk(z, k, 1)
    noise = 0.3 * torch.randn(rows, k, generator=g).double().cuda()
    logits = (zk - top + t * noise).float()
    d = (z - top) / t
    log_sum = torch.logsumexp(d, 1, keepdim=True)
    dk = (zk - top) / t
    logq = torch.log_softmax(logits.double() / t, 1)
    q = torch.exp(logq)
    want = torch.where(q > 0, q * (logq - dk + log_sum), 0.0).sum(1)
    a = (logits.double() / t).sub((logits.double() / t).amax(1, keepdim=True)).abs()
    each = q * ((2 * a + 10) * U * ((logq - dk + log_sum).abs() + 1)
                + 4 * U * (logq.abs() + dk.abs() + log_sum))
    tol = 2.0 ** -18 + 6 * U * (torch.exp(d - log_sum) * d.abs()).sum(1)
    tol += torch.where(q > 0, each, 0.0).sum(1)
    loss, lse = bo.linear_distillation(x, w, ids, logits, t)
    assert ((loss.double() - want).abs() <= tol).all(), ((loss.double() - want).abs() / tol).max()
    lse64 = (top / t + log_sum)[:, 0]
    assert ((lse.double() - lse64).abs() <= 2.0 ** -18 + 3 * U * lse64.abs()).all()


def test_minus_infinity_and_overflow(bo):
    """A word that the student rules out: an infinite loss where the teacher gives it,
    none where it does not."""
    for rows in (20, 200):
        x = torch.ones(rows, 8, device="cuda").bfloat16()
        w = torch.zeros(50, 8, device="cuda").bfloat16()
        w[7] = -3e38                              # the sum of eight: -inf
        w[9] = -1e38 / 8
        ids = torch.tensor([3, 4], device="cuda").repeat(rows, 1)
        ids[1, 0], ids[2, 0] = 7, 9
        loss, lse = bo.linear_distillation(x, w, ids, torch.zeros(rows, 2, device="cuda"))
        assert loss[1] == math.inf and loss[2] > 1e37
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[1:3] = False
        # 48 words of logit 0 and two that add nothing
        want = math.log(48) - math.log(2)
        assert ((loss[keep] - want).abs() <= 2.0 ** -18).all()
        assert ((lse - math.log(48)).abs() <= 2.0 ** -18).all()


@pytest.mark.parametrize("t,offset", [(1.0, 2048), (2.5, 2048), (0.05, 0), (0.05, 256)])
def test_gradients(bo, t, offset):
    """p is exp of a difference from the given lse: off by 2^-23 |lse| of itself (lse t,
    rounded), 6 u |d| + 2^-21 (factor, product, exponential), and q by (2 |a| + 10) u; one
    rounding of dz to 16 bits, at random, 4 h sqrt(sum dz^2 w^2); fp32 sums of `rows` or
    `vocab` products; and the result's own rounding."""
    g = torch.Generator().manual_seed(offset)
    rows, dim, vocab, k = 200, 64, 1000, 40
    x, w = eighths((rows, dim), g), eighths((vocab, dim), g)
    x[:, 0], w[:, 0] = offset / 64, 64 if offset else 0
    x, w = x.half().cuda(), w.half().cuda()
    t = float(torch.tensor(t).float())
    z = x.double() @ w.double().T
    zk, ids = torch.topk(z, k, 1)
    noise = 0.3 * torch.randn(rows, k, generator=g).double().cuda()
    logits = (zk - zk.amax(1, keepdim=True) + t * noise).float()
    dloss = (torch.rand(rows, generator=g) + 0.5).cuda() / rows
    _, lse = bo.linear_distillation(x, w, ids, logits, t)
    dx, dw = bo.linear_distillation_backward(dloss, x, w, ids, logits, lse, t)
    d = z / t - lse.double()[:, None]
    p, y = torch.exp(d), logits.double() / t
    q = torch.softmax(y, 1)
    arg = (y - y.amax(1, keepdim=True)).abs()
    r, r_off = (torch.zeros_like(p).scatter_add_(1, ids, v)
                for v in (q, q * (2 * arg + 10) * U))
    up = dloss.double()[:, None] / t
    dz = (p - r) * up
    off = (p * (2.0 ** -23 * lse.double().abs()[:, None] + 6 * U * d.abs() + 2.0 ** -21)
           + r_off) * up
    size, h = (p + r) * up, 2.0 ** -11
    for got, a, e, s, b in ((dx, dz, off, size, w.double()), (dw, dz.T, off.T, size.T, x.double())):
        ref = a @ b
        tol = 4 * h * (a.square() @ b.square()).sqrt()
        tol += e @ b.abs() + 4 * U * math.sqrt(a.shape[1]) * (s @ b.abs())
        tol += h * (ref.abs() + tol) + 2.0 ** -25
        assert ((got.double() - ref).abs() <= tol).all(), ((got.double() - ref).abs() / tol).max()
