"""The vocabulary's cross entropy (fp8_linear_xent and its gradient) on the
GPU against the definition in float64.

Tolerances, derived beforehand.  u = 2^-24 (fp32), h = the 16-bit type's unit
roundoff (2^-8 for bf16's 8 significant bits, 2^-11 for fp16's 11).  A logit is a sum of `dim` exact products in fp32; the
tensor core may drop bits below its alignment, so it is given
4 u * sqrt(dim) + 16 u of sum |x w| (a random walk with headroom).  loss and lse
are 1-Lipschitz in the logits (times 2 for the loss), plus the exponentials'
and sums' own error: 2^-20 absolute and 2^-22 relative.

dx and dw are held by 2-norms over the tensor: each element of p carries one
rounding of relative size at most h (the 16-bit type), so the error's norm is
at most h of the norm of the absolute products, sum |p| |w|, taken as a random
sum: 4 h * sqrt(sum p^2 w^2) per element, plus the result's own rounding, h of
the value, plus what the logits' and lse's error puts on p: |p| (3e-5).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}   # half the least spacing


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


def inputs(rows, dim, vocab, dtype, seed=0, ignored=0.2, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim, generator=g).to(dtype).cuda()
    w = (torch.randn(vocab, dim, generator=g) * spread / math.sqrt(dim)).to(dtype).cuda()
    t = torch.randint(0, vocab, (rows,), generator=g)
    t[torch.rand(rows, generator=g) < ignored] = -100
    dloss = torch.rand(rows, generator=g) + 0.5
    return x, w, t.cuda(), dloss.cuda()


def reference(x, w, t, dloss=None):
    z = x.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    live = t != -100
    loss = torch.where(live, lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    if dloss is None:
        return loss, lse
    p = torch.exp(z - lse[:, None])
    p[torch.arange(len(t), device=t.device), t.clamp(min=0)] -= 1
    p *= torch.where(live, dloss.double(), 0.0)[:, None]
    return p


def check_forward(bo, x, w, t, **kw):
    loss, lse = bo.linear_cross_entropy(x, w, t, **kw)
    loss64, lse64 = reference(x, w, t)
    dim = x.shape[1]
    top = (x.double().abs() @ w.double().abs().T).amax(1)
    tol = (4 * math.sqrt(dim) + 16) * U * top + 2.0 ** -20 + 2.0 ** -22 * lse64.abs()
    assert loss.dtype == lse.dtype == torch.float32
    assert (lse.double() - lse64).abs().le(tol).all()
    assert (loss.double() - loss64).abs().le(2 * tol).all()
    assert (loss[t == -100] == 0).all()
    return loss, lse


def check_backward(bo, x, w, t, dloss, lse=None, **kw):
    if lse is None:
        lse = reference(x, w, t)[1].float()
    dx, dw = bo.linear_cross_entropy_backward(dloss, x, w, t, lse, **kw)
    p = reference(x, w, t, dloss)
    h, tiny = HALF[x.dtype], TINY[x.dtype]
    for got, a, b in ((dx, p, w.double()), (dw, p.T, x.double())):
        ref = a @ b
        assert got.dtype == x.dtype and got.shape == ref.shape
        noise = (a.square() @ b.square()).sqrt()
        tol = 4 * h * noise + (3e-5 + 4 * U * math.sqrt(a.shape[1])) * (a.abs() @ b.abs())
        tol += h * (ref.abs() + tol) + tiny
        off = (got.double() - ref).abs() - tol
        assert off.le(0).all(), off.max()
    assert (dx[t == -100] == 0).all()
    return dx, dw


SIZES = [(1, 64, 1000), (3, 8, 1), (128, 64, 256), (129, 72, 257), (37, 768, 5003),
         (300, 200, 1031), (1025, 136, 2049), (256, 1024, 12000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,dim,vocab", SIZES)
def test_forward_and_backward(bo, rows, dim, vocab, dtype):
    x, w, t, dloss = inputs(rows, dim, vocab, dtype, seed=rows + vocab)
    check_forward(bo, x, w, t)
    check_backward(bo, x, w, t, dloss)


@pytest.mark.parametrize("rows", [1, 31, 33, 70, 128, 129, 256, 257])
def test_few_tokens_over_a_large_vocabulary(bo, rows):
    """More tiles of the vocabulary than pairs of SMs, for both ways of laying
    the tokens out, with targets at both ends and at tile borders."""
    x, w, t, dloss = inputs(rows, 64, 50257, torch.bfloat16, seed=rows, ignored=0.0)
    ends = torch.tensor([50256, 0, 255, 256, 50175, 50176, 31, 32], device="cuda")[:rows]
    t[:len(ends)] = ends
    check_forward(bo, x, w, t)
    if rows in (1, 129):
        check_backward(bo, x, w, t, dloss)


@pytest.mark.parametrize("dim", [1, 7, 65, 130])
def test_row_lengths_that_are_no_multiple_of_eight(bo, dim):
    x, w, t, dloss = inputs(70, dim, 301, torch.float16, seed=dim)
    check_forward(bo, x, w, t)
    check_backward(bo, x, w, t, dloss)


def test_unaligned_tensors(bo):
    x, w, t, dloss = inputs(70, 64, 301, torch.bfloat16, seed=5)
    shift = lambda a: torch.cat([a.new_zeros(1), a.reshape(-1)])[1:].view(a.shape)  # noqa: E731
    xs, ws = shift(x), shift(w)
    assert xs.data_ptr() % 16 and ws.data_ptr() % 16
    check_forward(bo, xs, ws, t)
    check_backward(bo, xs, ws, t, dloss)


def test_several_vocabulary_pieces(bo):
    # 4096 tokens: pieces of 8192 columns, the last one of 3 columns
    x, w, t, dloss = inputs(4096, 72, 8195, torch.bfloat16, seed=3)
    t[:5] = torch.tensor([0, 8191, 8192, 8194, 8193], device="cuda")
    check_forward(bo, x, w, t)
    check_backward(bo, x, w, t, dloss)


def test_ignored_tokens_may_hold_anything(bo):
    x, w, t, dloss = inputs(200, 64, 999, torch.float16, seed=7)
    clean_dx, clean_dw = check_backward(bo, x, w, t, dloss)
    lse = reference(x, w, t)[1].float()
    out = t == -100
    assert out.any() and not out.all()
    for bad in (float("nan"), float("inf"), -65504.0):
        xb, db, lb = x.clone(), dloss.clone(), lse.clone()
        xb[out], db[out], lb[out] = bad, bad, bad
        loss, _ = bo.linear_cross_entropy(xb, w, t)
        assert (loss[out] == 0).all() and torch.isfinite(loss).all()
        dx, dw = bo.linear_cross_entropy_backward(db, xb, w, t, lb)
        assert torch.equal(dx, clean_dx) and torch.equal(dw, clean_dw)


def test_every_token_ignored_and_no_token(bo):
    x, w, t, dloss = inputs(130, 64, 300, torch.bfloat16, ignored=2.0)
    loss, lse = check_forward(bo, x, w, t)
    dx, dw = bo.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    dx, dw = bo.linear_cross_entropy_backward(dloss[:0], x[:0], w, t[:0], lse[:0])
    assert dx.shape == (0, 64) and (dw == 0).all()
    loss, lse = bo.linear_cross_entropy(x[:0], w, t[:0])
    assert loss.numel() == lse.numel() == 0


def test_targets_outside_the_vocabulary_give_nan(bo):
    x, w, t, dloss = inputs(64, 64, 300, torch.bfloat16, ignored=0.0)
    t[3], t[9] = 300, -1
    loss, lse = bo.linear_cross_entropy(x, w, t)
    bad = torch.zeros_like(t, dtype=torch.bool)
    bad[3] = bad[9] = True
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all()
    dx, _ = bo.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[~bad]).all()


def test_ignore_index_inside_the_vocabulary(bo):
    x, w, t, _ = inputs(64, 64, 300, torch.bfloat16, ignored=0.0)
    t[::4] = 17
    loss, _ = bo.linear_cross_entropy(x, w, t, ignore_index=17)
    assert (loss[::4] == 0).all() and (loss[1::4] > 0).all()


def test_far_logits(bo):
    # one certain token and logits of some thousands: the maximum is taken off
    x, w, t, dloss = inputs(40, 64, 600, torch.bfloat16, seed=2, spread=300.0, ignored=0.0)
    t[:20] = (x[:20].double() @ w.double().T).argmax(1)
    check_forward(bo, x, w, t)


def test_small_and_large_loss_scales_in_fp16(bo):
    # powers of two of dloss scale the result exactly, as far as FP16 holds it
    x, w, t, dloss = inputs(100, 64, 700, torch.float16, seed=4)
    lse = reference(x, w, t)[1].float()
    dx, dw = check_backward(bo, x, w, t, dloss, lse)
    for k in (2.0 ** 10, 2.0 ** -6):
        dxk, dwk = bo.linear_cross_entropy_backward(dloss * k, x, w, t, lse)
        for a, b in ((dx, dxk), (dw, dwk)):
            big = (a.double() * k).abs().ge(2.0 ** -14) & a.double().abs().ge(2.0 ** -14)
            assert torch.equal((a.double() * k)[big], b.double()[big])


def test_same_bits_every_time_and_on_another_stream(bo):
    x, w, t, dloss = inputs(500, 128, 3001, torch.bfloat16, seed=9)
    first = None
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(4):
        stream = side if k % 2 else None
        loss, lse = bo.linear_cross_entropy(x, w, t, stream=stream)
        dx, dw = bo.linear_cross_entropy_backward(dloss, x, w, t, lse, stream=stream)
        torch.cuda.synchronize()
        got = [loss, lse, dx, dw]
        first = first or [a.clone() for a in got]
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_gradient_against_differences(bo):
    """The slope of the float64 loss along random directions against the
    kernel's gradients: the central difference's error is O(step^2)."""
    x, w, t, dloss = inputs(48, 64, 500, torch.float16, seed=6)
    _, lse = bo.linear_cross_entropy(x, w, t)
    dx, dw = bo.linear_cross_entropy_backward(dloss, x, w, t, lse)
    g = torch.Generator().manual_seed(1)
    step = 1e-4
    for a, grad, other in ((x, dx, 0), (w, dw, 1)):
        d = torch.randn(a.shape, generator=g).double().cuda()
        f = lambda s: (reference(x.double() + (s * d if other == 0 else 0),  # noqa: E731
                                 w.double() + (s * d if other == 1 else 0), t)[0]
                       * dloss.double()).sum()
        slope = (f(step) - f(-step)) / (2 * step)
        got = (grad.double() * d).sum()
        # each element's error is below 5 h of a random sum of its size
        tol = 8 * HALF[torch.float16] * grad.double().norm() + 1e-5 * slope.abs()
        assert (got - slope).abs() <= tol


def test_captured_in_a_graph(bo):
    x, w, t, dloss = inputs(200, 128, 1500, torch.bfloat16, seed=11)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        loss, lse = bo.linear_cross_entropy(x, w, t)
        dx, dw = bo.linear_cross_entropy_backward(dloss, x, w, t, lse)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        loss2, lse2 = bo.linear_cross_entropy(x, w, t)
        dx2, dw2 = bo.linear_cross_entropy_backward(dloss, x, w, t, lse2)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, loss2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    del g
    bo.release_stream(s)


def test_refusals(bo):
    x, w, t, dloss = inputs(8, 64, 100, torch.bfloat16)
    lse = torch.zeros(8, device="cuda")
    f, b = bo.linear_cross_entropy, bo.linear_cross_entropy_backward
    with pytest.raises(TypeError):
        f(x.float(), w.float(), t)
    with pytest.raises(TypeError):
        f(x, w.half(), t)
    with pytest.raises(TypeError):
        f(x, w, t.int())
    with pytest.raises(TypeError):
        f(x.cpu(), w, t)
    with pytest.raises(ValueError):
        f(x, w[:, :56].contiguous(), t)
    with pytest.raises(ValueError):
        f(x.T.contiguous().T, w, t)
    with pytest.raises(ValueError):
        f(x, w, t[:7])
    with pytest.raises(ValueError):
        f(x[None], w, t)
    with pytest.raises(TypeError):
        b(dloss.double(), x, w, t, lse)
    with pytest.raises(ValueError):
        b(dloss[:5], x, w, t, lse)
