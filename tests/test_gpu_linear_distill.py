"""Distillation from a teacher's top logits (fp8_linear_distill and its gradient)
against the definition in float64.

Tolerances, derived beforehand, as the cross entropy's (test_gpu_linear_xent.py): u
= 2^-24, h = half a step of the 16-bit type.  A logit is given (4 sqrt(dim) + 16) u
of sum |x w|, lse and loss 2^-20 absolute and 2^-22 relative besides, logits divided
by the temperature t.  The teacher's shares q are exponentials of an argument a =
(l - max l) / t: off by (2 |a| + 10) u of themselves, which the loss meets times
|log q - log p| + 1; its terms' own roundings are 8 u of |log q| + |z / t| + |lse|.

dx and dw: one rounding of dz to 16 bits per element, at random, 4 h sqrt(sum dz^2
w^2); what the logits, lse and q are off by, 3e-5 max(1, 1 / t) of p and q (which
cancel in dz); and the result's own rounding.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


def inputs(rows, dim, vocab, k, dtype, ldtype=F, seed=0, none=0.2, missing=0.2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim, generator=g).to(dtype).cuda()
    w = (torch.randn(vocab, dim, generator=g) * 1.5 / math.sqrt(dim)).to(dtype).cuda()
    ids = torch.randint(0, vocab, (rows, k), generator=g)       # (some words twice)
    near = torch.rand(rows, k, generator=g) < 0.5               # frequent words first
    ids = torch.where(near, ids % min(vocab, 300), ids)
    ids[torch.rand(rows, k, generator=g) < missing] = -1
    ids[torch.rand(rows, generator=g) < none] = -100
    logits = (3 * torch.randn(rows, k, generator=g)).to(ldtype)
    dloss = torch.rand(rows, generator=g) + 0.5
    return x, w, ids.cuda(), logits.cuda(), dloss.cuda()


def teacher(ids, logits, t):
    """log q, q (0 where an entry does not count) and whether a token has any."""
    y = torch.where(ids >= 0, logits.double() / t, -math.inf)
    live = (y > -math.inf).any(1)
    y = y - y.amax(1, keepdim=True)      # (near fp32's lowest number, y + log 10 is y)
    logq = y - torch.logsumexp(y, 1, keepdim=True)
    q = torch.where((y > -math.inf) & live[:, None], torch.exp(logq), 0.0)
    return torch.where(q > 0, logq, 0.0), q, live


def check_forward(bo, x, w, ids, logits, t):
    loss, lse = bo.linear_distillation(x, w, ids, logits, t)
    t = float(torch.tensor(t).float())
    logq, q, live = teacher(ids, logits, t)
    z = x.double() @ w.double().T / t
    lse64 = torch.logsumexp(z, 1)
    zk = z.gather(1, ids.clamp(min=0))
    loss64 = (q * (logq - zk + lse64[:, None])).sum(1)
    top = (x.double().abs() @ w.double().abs().T).amax(1) / t
    tol = (4 * math.sqrt(x.shape[1]) + 16) * U * top + 2.0 ** -20 + 2.0 ** -22 * lse64.abs()
    assert loss.dtype == lse.dtype == F
    assert (lse.double() - lse64).abs().le(tol).all()
    a = logits.double() / t
    a = (a - torch.where(q > 0, a, -math.inf).amax(1, keepdim=True)).abs()
    off = q * ((2 * a + 10) * U * ((logq - zk + lse64[:, None]).abs() + 1)
               + 8 * U * (logq.abs() + zk.abs() + lse64.abs()[:, None]))
    off = torch.where(q > 0, off, 0.0).sum(1)
    assert (loss.double() - loss64).abs().le(2 * tol + off).all()
    assert (loss[~live] == 0).all()
    again = bo.linear_distillation(x, w, ids, logits, t)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    return loss, lse


def check_backward(bo, x, w, ids, logits, t, dloss):
    lse = torch.logsumexp(x.double() @ w.double().T / t, 1).float()
    dx, dw = bo.linear_distillation_backward(dloss, x, w, ids, logits, lse, t)
    t = float(torch.tensor(t).float())
    _, q, live = teacher(ids, logits, t)
    p = torch.exp(x.double() @ w.double().T / t - lse.double()[:, None])
    r = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), q)
    g = torch.where(live, dloss.double() / t, 0.0)[:, None]
    dz, size = (p - r) * g, (p + r) * g.abs()
    h, tiny = HALF[x.dtype], TINY[x.dtype]
    for got, a, s, b in ((dx, dz, size, w.double()), (dw, dz.T, size.T, x.double())):
        ref = a @ b
        assert got.dtype == x.dtype and got.shape == ref.shape
        tol = 4 * h * (a.square() @ b.square()).sqrt()
        tol += (3e-5 * max(1, 1 / t) + 4 * U * math.sqrt(a.shape[1])) * (s @ b.abs())
        tol += h * (ref.abs() + tol) + tiny
        off = (got.double() - ref).abs() - tol
        assert off.le(0).all(), off.max()
    assert (dx[~live] == 0).all()
    return dx, dw


SIZES = [(1, 64, 1000, 1), (3, 8, 1, 2), (128, 64, 256, 7), (129, 72, 257, 33), (37, 768, 5003, 64),
         (300, 200, 1031, 256), (1025, 136, 2049, 20), (256, 1024, 12000, 100)]


@pytest.mark.parametrize("dtype,ldtype,t", [(BF, F, 1.0), (HF, BF, 2.5), (HF, HF, 0.5)])
@pytest.mark.parametrize("rows,dim,vocab,k", SIZES)
def test_forward_and_backward(bo, rows, dim, vocab, k, dtype, ldtype, t):
    args = inputs(rows, dim, vocab, k, dtype, ldtype, seed=rows + vocab)
    check_forward(bo, *args[:4], t)
    check_backward(bo, *args[:4], t, args[4])


@pytest.mark.parametrize("rows", [1, 31, 33, 70, 128, 129, 257])
def test_words_at_the_ends_of_tiles(bo, rows):
    x, w, ids, logits, dloss = inputs(rows, 64, 50257, 64, BF, seed=rows, none=0.0)
    ends = torch.tensor([50256, 0, 255, 256, 127, 128, 50175, 50176, 31, 32, 95, 96, 383, 384,
                         -1, 511, 512, 129, 1], device="cuda")
    ids[:, 5:5 + len(ends)] = ends
    check_forward(bo, x, w, ids, logits, 1.0)
    if rows in (1, 33, 257):
        check_backward(bo, x, w, ids, logits, 1.0, dloss)


@pytest.mark.parametrize("rows", [40, 200])
def test_all_entries_in_one_tile(bo, rows):
    """Every word of a tile an entry of every token; a word 256 times."""
    x, w, ids, logits, dloss = inputs(rows, 64, 1000, 256, HF, seed=2, none=0.0, missing=0.0)
    for first in (0, 256, 744):
        ids[:] = torch.randperm(256, device="cuda") + first
        ids[3] = first + 17
        ids[4, ::2] = first
        check_forward(bo, x, w, ids, logits, 1.0)
        check_backward(bo, x, w, ids, logits, 1.0, dloss)


@pytest.mark.parametrize("dim", [1, 7, 65, 130])
def test_row_lengths_that_are_no_multiple_of_eight(bo, dim):
    args = inputs(70, dim, 301, 9, HF, seed=dim)
    check_forward(bo, *args[:4], 1.5)
    check_backward(bo, *args[:4], 1.5, args[4])


def test_unaligned_tensors(bo):
    x, w, ids, logits, dloss = inputs(200, 64, 301, 5, BF, BF, seed=5)
    shift = lambda a: torch.cat([a.new_zeros(1), a.reshape(-1)])[1:].view(a.shape)  # noqa: E731
    x, w, ids, logits, dloss = (shift(a) for a in (x, w, ids, logits, dloss))
    check_forward(bo, x, w, ids, logits, 1.0)
    check_backward(bo, x, w, ids, logits, 1.0, dloss)


def test_several_vocabulary_pieces(bo):
    # 4096 tokens: pieces of 8192 columns, the last one of 3 columns
    x, w, ids, logits, dloss = inputs(4096, 72, 8195, 16, BF, seed=3)
    ids[:, 0], ids[:, 1], ids[:, 2], ids[:, 3] = 8191, 8192, 8194, 8193
    check_forward(bo, x, w, ids, logits, 1.0)
    check_backward(bo, x, w, ids, logits, 1.0, dloss)


def test_more_tokens_than_one_launch(bo):
    x, w, ids, logits, dloss = inputs(65536 + 300, 16, 700, 6, HF, seed=1)
    check_forward(bo, x, w, ids, logits, 1.0)
    check_backward(bo, x, w, ids, logits, 1.0, dloss)


def test_a_student_that_agrees(bo):
    """The teacher is the student, all of its words: p - q is what 16-bit logits
    leave of nothing, and the gradient with it."""
    x, w, ids, logits, dloss = inputs(150, 64, 200, 200, HF, seed=8, none=0.0)
    ids[:] = torch.arange(200, device="cuda")
    logits = (x.double() @ w.double().T).float()
    loss, _ = check_forward(bo, x, w, ids, logits, 2.0)
    dx, _ = check_backward(bo, x, w, ids, logits, 2.0, dloss)
    assert loss.abs().max() < 1e-5 and dx.abs().max() < 1e-5


def test_one_word_is_the_cross_entropy(bo):
    """One entry a token: the cross entropy of its word, and its gradients."""
    for rows in (60, 300):
        x, w, ids, logits, dloss = inputs(rows, 72, 901, 1, BF, seed=rows, missing=0.0)
        loss, lse = bo.linear_distillation(x, w, ids, logits)
        target = torch.where(ids[:, 0] >= 0, ids[:, 0], -100)
        want, lse2 = bo.linear_cross_entropy(x, w, target)
        assert torch.equal(lse, lse2)
        assert ((loss - want).abs() <= 4 * U * (lse.abs() + want.abs() + 10)).all()
        got = bo.linear_distillation_backward(dloss, x, w, ids, logits, lse)
        ref = bo.linear_cross_entropy_backward(dloss, x, w, target, lse)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_tokens_without_a_teacher_may_hold_anything(bo):
    x, w, ids, logits, dloss = inputs(300, 64, 999, 12, HF, seed=7)
    dead = (ids < 0).all(1)
    assert dead.any() and not dead.all()
    lse = torch.logsumexp(x.double() @ w.double().T, 1).float()
    clean = bo.linear_distillation_backward(dloss, x, w, ids, logits, lse)
    loss, _ = bo.linear_distillation(x, w, ids, logits)
    x, logits, dloss, lse = x.clone(), logits.clone(), dloss.clone(), lse.clone()
    x[dead], logits[dead], dloss[dead], lse[dead] = math.nan, math.nan, math.inf, math.nan
    logits[ids < 0] = math.nan               # an entry that is not given
    loss2, _ = bo.linear_distillation(x, w, ids, logits)
    assert torch.equal(loss, loss2)
    again = bo.linear_distillation_backward(dloss, x, w, ids, logits, lse)
    assert torch.equal(clean[0], again[0]) and torch.equal(clean[1], again[1])


def test_entries_of_minus_infinity_do_not_count(bo):
    x, w, ids, logits, dloss = inputs(200, 64, 400, 10, BF, seed=9, none=0.0, missing=0.0)
    off = torch.rand(200, 10, device="cuda") < 0.4
    off[5] = True                            # a token with nothing left
    gone = ids.masked_fill(off, -1)
    logits[off] = -math.inf
    check_forward(bo, x, w, ids, logits, 1.0)
    a = bo.linear_distillation(x, w, ids, logits)
    b = bo.linear_distillation(x, w, gone, logits)
    assert torch.equal(a[0], b[0]) and a[0][5] == 0
    a = bo.linear_distillation_backward(dloss, x, w, ids, logits, a[1])
    b = bo.linear_distillation_backward(dloss, x, w, gone, logits, b[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and (a[0][5] == 0).all()
    # the lowest number is one like any other
    logits[off] = torch.finfo(F).min
    check_forward(bo, x, w, ids, logits, 1.0)


@pytest.mark.parametrize("rows", [20, 200])
def test_what_spoils_a_token(bo, rows):
    x, w, ids, logits, dloss = inputs(rows, 64, 400, 10, BF, seed=9, none=0.0, missing=0.0)
    good, lse = bo.linear_distillation(x, w, ids, logits)
    ids[0, 3], ids[1, 0], ids[2, 9] = 400, 2 ** 40, -2 ** 50      # the last is not given
    logits[3, 2], logits[4, 1] = math.nan, math.inf
    loss, lse2 = bo.linear_distillation(x, w, ids, logits)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[0, 1, 3, 4]] = True
    assert loss[bad].isnan().all() and torch.equal(lse, lse2)
    keep = ~bad
    keep[2] = False
    assert torch.equal(loss[keep], good[keep]) and loss[2].isfinite()
    dx, dw = bo.linear_distillation_backward(dloss, x, w, ids, logits, lse)
    assert dx[bad].isnan().all() and dx[~bad].isfinite().all() and dw.isnan().all()


def test_small_dloss_keeps_its_gradient(bo):
    x, w, ids, logits, dloss = inputs(300, 64, 700, 8, HF, seed=4)
    dloss[::3] *= 2.0 ** -20
    lse = torch.logsumexp(x.double() @ w.double().T, 1).float()
    dx, _ = bo.linear_distillation_backward(dloss * 1024, x, w, ids, logits, lse)
    _, q, live = teacher(ids, logits, 1.0)
    p = torch.exp(x.double() @ w.double().T - lse.double()[:, None])
    p.scatter_add_(1, ids.clamp(min=0), -q)
    ref = (p * (dloss * 1024 * live).double()[:, None]) @ w.double()
    small = ref[::3]
    assert (dx[::3].double() - small).norm() <= 2.0 ** -9 * small.norm() + 2.0 ** -25 * 64


def test_empty(bo):
    x = torch.zeros(0, 64, dtype=BF, device="cuda")
    w = torch.randn(30, 64, device="cuda").to(BF)
    ids = torch.zeros(0, 4, dtype=torch.long, device="cuda")
    loss, lse = bo.linear_distillation(x, w, ids, ids.float())
    assert loss.shape == lse.shape == (0,)
    dx, dw = bo.linear_distillation_backward(loss, x, w, ids, ids.float(), lse)
    assert dx.shape == (0, 64) and dw.eq(0).all()


def test_captured_beside_the_cross_entropy(bo):
    """Both in one graph, on one stream's scratch, with new inputs at each replay."""
    s = torch.cuda.Stream()
    x, w, ids, logits, dloss = inputs(300, 64, 3000, 16, BF, seed=1)
    target = ids[:, 0].clamp(min=0).contiguous()

    def both():
        a = bo.linear_distillation(x, w, ids, logits, 2.0)
        b = bo.linear_distillation_backward(dloss, x, w, ids, logits, a[1], 2.0)
        c = bo.linear_cross_entropy(x, w, target)
        d = bo.linear_cross_entropy_backward(dloss, x, w, target, c[1])
        return a + b + c + d
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = both()
    for seed in (2, 3):
        for a, b in zip((x, w, ids, logits, dloss), inputs(300, 64, 3000, 16, BF, seed=seed)):
            a.copy_(b)
        target.copy_(ids[:, 0].clamp(min=0))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, both()):
            assert torch.equal(a, b)
    del g
    bo.release_stream(s)


def test_autograd(bo):
    from bit_optimizer_gb300 import nn
    x, w, ids, logits, _ = inputs(120, 64, 500, 20, HF, seed=6)
    x = x.view(4, 30, 64).requires_grad_(True)
    w.requires_grad_(True)
    ids, logits = ids.view(4, 30, 20), logits.view(4, 30, 20)
    xd, wd = (a.detach().double().requires_grad_(True) for a in (x, w))
    logq, q, live = teacher(ids.view(-1, 20), logits.view(-1, 20), 2.0)
    logp = torch.log_softmax(xd.view(-1, 64) @ wd.T / 2, 1).gather(1, ids.view(-1, 20).clamp(min=0))
    each = (q * (logq - logp)).sum(1)
    for reduction, want in (("none", each.view(4, 30)), ("sum", each.sum()),
                            ("mean", each.sum() / live.sum())):
        loss = nn.linear_distillation(x, w, ids, logits, 2.0, reduction)
        assert loss.shape == want.shape and (loss.double() - want).abs().max() < 1e-4
        if reduction == "none":
            continue
        got = torch.autograd.grad(loss * 64, (x, w))
        ref = torch.autograd.grad(want * 64, (xd, wd), retain_graph=True)
        for a, b in zip(got, ref):
            assert (a.double() - b).norm() <= 2.0 ** -10 * b.norm()
    # against differences, in the direction of the gradient
    dx, = torch.autograd.grad(nn.linear_distillation(x, w, ids, logits, 2.0, "sum"), x)
    step = 2.0 ** -6 * torch.sign(dx.float()).half()
    up, down = (nn.linear_distillation((x + k * step).detach(), w, ids, logits, 2.0, "sum")
                for k in (1, -1))
    moved = ((x + step).double() - (x - step).double()).detach()
    slope = (dx.double() * moved).sum()
    assert abs((up - down).double() - slope) <= 1e-2 * slope
    # nothing left: no loss, no gradient
    loss = nn.linear_distillation(x, w, torch.full_like(ids, -1), logits)
    dx, dw = torch.autograd.grad(loss, (x, w))
    assert loss == 0 and dx.eq(0).all() and dw.eq(0).all()


def test_refusals(bo):
    x, w, ids, logits, dloss = inputs(10, 64, 50, 4, BF)
    cases = [(TypeError, lambda: bo.linear_distillation(x.float(), w, ids, logits)),
             (TypeError, lambda: bo.linear_distillation(x, w.half(), ids, logits)),
             (TypeError, lambda: bo.linear_distillation(x, w, ids.int(), logits)),
             (TypeError, lambda: bo.linear_distillation(x, w, ids, logits.double())),
             (ValueError, lambda: bo.linear_distillation(x, w, ids[:5], logits[:5])),
             (ValueError, lambda: bo.linear_distillation(x, w, ids, logits[:, :3])),
             (ValueError, lambda: bo.linear_distillation(x, w, ids[:, :3], logits[:, :3])),
             (ValueError, lambda: bo.linear_distillation(x, w, ids[:, :0], logits[:, :0])),
             (ValueError, lambda: bo.linear_distillation(x, w, ids.repeat(1, 65),
                                                         logits.repeat(1, 65))),
             (ValueError, lambda: bo.linear_distillation_backward(dloss[:5], x, w, ids, logits,
                                                                  dloss))]
    for t in (0.0, -1.0, math.nan, math.inf):
        cases.append((bo.Fp8OptError, lambda t=t: bo.linear_distillation(x, w, ids, logits, t)))
    for error, call in cases:
        with pytest.raises(error):
            call()
