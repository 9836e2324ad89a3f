"""The cross entropy where its numbers are far apart, against the definition in
float64.

Tolerances, derived beforehand, as in test_gpu_linear_xent.py: h the type's unit
roundoff, u = 2^-24.  An element of p is rounded once, by at most h of itself or,
where FP16 becomes subnormal, by 2^-25; p is held at no less than 2^2 (a factor
in [1, 2^15] of 2^15 for a token within 2^12 of the largest dloss, [2^2, 2^3] for
any other), so by at most 2^-27 of the token's dloss.  Rounding errors of a sum
are taken as a random sum with a factor of 4.  dw reads rows of x scaled by 2^-b,
subnormal below 2^-14: off by 2^-25, in a product with p of at most 2^3 out of
2^15: 2^-37 of the largest dloss times p of the token's own.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


@pytest.mark.parametrize("dtype,span", [(torch.float16, 30), (torch.bfloat16, 60)])
@pytest.mark.parametrize("rows,dim,vocab", [(100, 64, 700), (310, 65, 5003), (129, 136, 257)])
def test_loss_gradients_far_apart(bo, rows, dim, vocab, dtype, span):
    """Tokens whose dloss differ by up to 2^span: each token's dx is as near as
    if it were alone."""
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, dim, generator=g).to(dtype).cuda()
    w = (torch.randn(vocab, dim, generator=g) * 1.5 / math.sqrt(dim)).to(dtype).cuda()
    t = torch.randint(0, vocab, (rows,), generator=g).cuda()
    e = torch.arange(rows) * 7 % (span + 1)
    dloss = (torch.rand(rows, generator=g) + 1) * torch.exp2(13.0 - e)
    dloss = torch.where(torch.arange(rows) % 3 == 0, -dloss, dloss).cuda()
    dloss[5] = 0
    t[7], dloss[7] = -100, float("inf")
    x[7] = float("nan")
    xr = torch.where((t == -100)[:, None], torch.zeros_like(x), x).double()
    z = xr @ w.double().T
    lse = torch.logsumexp(z, 1)
    dx, dw = bo.linear_cross_entropy_backward(dloss, x, w, t, lse.float())
    q = torch.exp(z - lse[:, None])
    q[torch.arange(rows, device="cuda"), t.clamp(min=0)] -= 1
    d = torch.where(t == -100, torch.zeros_like(dloss), dloss).double()
    p, h = q * d[:, None], HALF[dtype]
    assert (dx[5] == 0).all() and (dx[7] == 0).all()
    top = d.abs().max()
    for got, a, b, own in (
            (dx, p, w.double(), 2.0 ** -27 * d.abs()[:, None] * w.double().square().sum(0).sqrt()),
            (dw, p.T, xr, 2.0 ** -27 * (d.square() @ xr.square()).sqrt()
             + 2.0 ** -37 * top * q.abs().sum(0)[:, None])):
        ref = a @ b
        tol = 4 * h * (a.square() @ b.square()).sqrt() + 4 * own
        tol += (3e-5 + 4 * U * math.sqrt(a.shape[1])) * (a.abs() @ b.abs())
        tol += h * (ref.abs() + tol) + TINY[dtype]
        off = (got.double() - ref).abs() - tol
        assert off.le(0).all(), off.max()


@pytest.mark.parametrize("rows", [5, 128, 300])
def test_logits_near_the_ends_of_fp32(bo, rows):
    """Tokens whose logits are all far below zero, above it, or minus infinity.
    A logit is 8 products of powers of two, exact in fp32, so lse is off by its
    logarithm's and sums' 2^-22 relative and 2^-20 absolute."""
    dim, vocab = 8, 700
    scale = torch.exp2(torch.arange(rows) % 5 * 30.0 - 60)          # 2^-60 .. 2^60
    x = scale[:, None].expand(rows, dim).to(torch.bfloat16).cuda()
    w = -torch.exp2(torch.arange(vocab) % 9 + 52.0)                 # -2^52 .. -2^60
    w = w[:, None].expand(vocab, dim).to(torch.bfloat16).cuda()
    t = torch.arange(rows, device="cuda") * 9 % vocab               # the largest logits
    for sign in (1, -1):
        z = (x.double() @ (sign * w.double()).T)
        assert z.abs().max() > 1e36 and z.abs().max() < 3e38
        lse64 = torch.logsumexp(z, 1)
        loss64 = lse64 - z.gather(1, t[:, None])[:, 0]
        loss, lse = bo.linear_cross_entropy(x, sign * w, t)
        assert ((lse.double() - lse64).abs() <= 2.0 ** -20 + 2.0 ** -22 * lse64.abs()).all()
        assert ((loss.double() - loss64).abs()
                <= 2.0 ** -19 + 2.0 ** -21 * (lse64.abs() + loss64)).all()
    # logits of minus infinity beside finite ones, and nothing else
    one = torch.ones(rows, dim, dtype=torch.bfloat16, device="cuda")
    w[::3] = float("-inf")
    w[1::3], w[2::3] = 0.5, -0.25
    t = torch.full((rows,), 1, device="cuda")
    loss, lse = bo.linear_cross_entropy(one, w, t)
    z = torch.where(torch.isinf(w[:, 0]), w[:, 0].double(), 8 * w[:, 0].double())
    assert ((lse.double() - torch.logsumexp(z, 0)).abs() <= 2.0 ** -19).all()
    assert ((loss.double() - (torch.logsumexp(z, 0) - 4)).abs() <= 2.0 ** -18).all()
    w[:] = float("-inf")
    assert (bo.linear_cross_entropy(one, w, t)[1] == float("-inf")).all()
