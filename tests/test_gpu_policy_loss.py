"""The clipped policy loss and its gradient against the definition in 64 bits and
against differences of it: every form of advantage, mask, reference and mean,
lengths from one token on, in and off vectors of four."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def package():
    global bo, nn
    import bit_optimizer_gb300 as bo
    from bit_optimizer_gb300 import nn


U = 2.0 ** -24      # half a step of fp32


def make(batch, length, per_token, ref, masked, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * length)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)
    lp = -torch.exp(randn(batch, length))
    old = lp + 0.25 * randn(batch, length)
    mask = None
    if masked:
        mask = torch.rand(batch, length, device="cuda", generator=g) < 0.7
        mask[::3] = False                               # sequences without a token
        old = torch.where(mask, old, torch.full_like(old, -math.inf))
    refp = lp + 0.6 * randn(batch, length) if ref else None
    if masked and ref:
        refp = torch.where(mask, refp, torch.full_like(refp, math.nan))
    adv = randn(batch, length) if per_token else randn(batch)
    return lp, old, adv, mask, refp


def terms(lp, old, adv, mask, refp, low, high, kl_coef):
    """Per token in fp64: policy term, KL, clipped, derivative, and bounds of the
    fp32 errors of the first two and the last."""
    lp, old = lp.double(), old.double()
    a = (adv if adv.dim() == 2 else adv[:, None].expand_as(lp)).double()
    on = torch.ones_like(lp, dtype=torch.bool) if mask is None else mask
    zero = torch.zeros_like(lp)
    d = torch.where(on, lp - old, zero)
    r = torch.exp(d)
    held = r.clamp(1 - low, 1 + high)
    clipped = (held * a < r * a) & on
    policy = torch.where(clipped, -held * a, -r * a) * on
    e = zero if refp is None else torch.where(on, refp.double() - lp, zero)
    kl = torch.expm1(e) - e
    slope = (torch.where(clipped, zero, -r * a) - kl_coef * torch.expm1(e)) * on
    # the difference's rounding, an exponential of 2 units, a product, the border's
    # own rounding
    err_policy = (d.abs() + 6) * (r * a).abs() * U * on
    # the difference's rounding through the derivative, ten steps of the series, and
    # beyond 1 an exponential and two sums
    wide = (e.abs() > 1) * (torch.exp(e) + 1 + e.abs())
    err_kl = (torch.expm1(e).abs() * e.abs() + 14 * kl + 4 * wide) * U
    err_slope = err_policy + abs(kl_coef) * (
        (torch.exp(e) * e.abs() + 14 * kl + e.abs() + 2 * torch.expm1(e).abs() + 4 * wide) * U)
    return policy, kl, clipped, slope, err_policy, err_kl, err_slope, on


def weights(on, by_sequence):
    n = on.sum(1).double()
    w = torch.where(n > 0, 1 / (n * (n > 0).sum()) if by_sequence else 1 / n.sum(), 0.0)
    return torch.nan_to_num(w)


def check(args, low=0.2, high=0.2, kl_coef=0.1, reduction="token"):
    lp, old, adv, mask, refp = args
    policy, kl, clipped, slope, ep, ek, es, on = terms(*args, low, high, kl_coef)
    w = weights(on, reduction == "sequence")
    stats, weight = bo.policy_loss(lp, old, adv, mask, refp, low, high, kl_coef, reduction)
    assert stats.shape == (4,) and weight.shape == lp.shape[:1]
    assert ((weight.double() - w).abs() <= U * w).all()
    means = [(t * w[:, None]).sum() for t in (policy, kl, clipped)]
    # a lane adds at most 32 terms in fp32; the rest is fp64
    bounds = [((e + 32 * U * t.abs()) * w[:, None]).sum() for t, e in
              ((policy, ep), (kl, ek), (clipped * 0.0, 0.0 * ep))]
    for got, want, b in zip(stats[1:].double(), means, bounds):
        assert (got - want).abs() <= b + 2 * U * want.abs() + 1e-30
    want = means[0] + kl_coef * means[1]
    assert (stats[0].double() - want).abs() <= (bounds[0] + abs(kl_coef) * bounds[1]
                                               + 2 * U * want.abs() + 1e-30)
    dloss = torch.tensor(1.7, device="cuda")
    d = bo.policy_loss_backward(dloss, lp, old, adv, weight, mask, refp, low, high, kl_coef)
    g = 1.7 * w[:, None]
    want = slope * dloss.double() * w[:, None]
    assert ((d.double() - want).abs() <= es * g * 1.01 + 6 * U * (slope.abs() * g) + 1e-37).all()
    if mask is not None:
        assert d[~mask].eq(0).all()
    again = bo.policy_loss(lp, old, adv, mask, refp, low, high, kl_coef, reduction)
    assert torch.equal(again[0], stats) and torch.equal(again[1], weight)
    return stats, d


SHAPES = [(1, 1), (3, 1), (1, 5), (2, 64), (5, 127), (4, 1024), (3, 1025), (2, 4100), (1, 40001),
          (700, 12), (5000, 3), (1, 70000), (40, 2048)]


@pytest.mark.parametrize("batch,length", SHAPES)
@pytest.mark.parametrize("per_token,ref,masked", [(False, True, True), (True, True, False),
                                                  (True, False, True), (False, False, False)])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_loss_and_gradient(batch, length, per_token, ref, masked, reduction):
    check(make(batch, length, per_token, ref, masked), reduction=reduction)


@pytest.mark.parametrize("low,high,kl", [(0.0, 0.0, 0.0), (1.0, math.inf, 0.5), (0.1, 0.3, -0.2),
                                         (1.0, 0.0, 3.0)])
def test_borders(low, high, kl):
    check(make(6, 500, True, True, True, 3), low, high, kl, "sequence")


def test_tokens_at_the_border():
    """Ratios within a few roundings of 1 + high and 1 - low, on either side: which
    are clipped follows from the exact difference."""
    n = 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    lp = -torch.exp(torch.randn(2, n, device="cuda", generator=g))
    border = torch.tensor([math.log(1.2), math.log(0.8)], device="cuda", dtype=torch.float64)
    old = (lp.double() - border[:, None]).float()
    step = torch.randint(-3, 4, (2, n), device="cuda", generator=g)
    old = (old.view(torch.int32) + step.int()).view(torch.float32)
    adv = torch.tensor([1.0, -1.0], device="cuda")
    stats, d = check((lp, old, adv, None, None), 0.2, 0.2, 0.0)
    assert 0.2 < stats[3] < 0.8 and d.eq(0).double().mean() == stats[3].double()


def test_small_kl_keeps_its_digits():
    lp = -torch.rand(8, 400, device="cuda", dtype=torch.float64).float() - 1
    ref = lp + 1e-3 * torch.randn(8, 400, device="cuda")
    args = (lp, lp.clone(), torch.zeros(8, device="cuda"), None, ref)
    stats, _ = check(args, kl_coef=1.0)
    e = ref.double() - lp.double()
    want = (e * e / 2 + e ** 3 / 6 + e ** 4 / 24).mean()
    assert (stats[2].double() - want).abs() <= 1e-5 * want


def test_against_differences():
    args = make(4, 30, False, True, True, 5)
    lp, old, adv, mask, refp = args
    _, d = check(args, reduction="sequence", kl_coef=0.3)
    h = 1e-5                                             # in fp64

    def loss(x):
        policy, kl, *_ = terms(x, old, adv, mask, refp, 0.2, 0.2, 0.3)
        return ((policy + 0.3 * kl) * weights(mask, True)[:, None]).sum()
    for b, t in [(1, 3), (1, 8), (2, 0), (2, 29), (0, 4)]:
        up, down = lp.double().clone(), lp.double().clone()
        up[b, t] += h
        down[b, t] -= h
        slope = (loss(up) - loss(down)) / (2 * h) * 1.7
        assert abs(slope - d[b, t].double()) <= 1e-4 * abs(slope) + 1e-7


def test_nothing_left():
    lp, old, adv, mask, refp = make(5, 40, False, True, True)
    mask = torch.zeros_like(mask)
    for reduction in ("token", "sequence"):
        stats, weight = bo.policy_loss(lp, old, adv, mask, refp, kl_coef=1.0,
                                       reduction=reduction)
        assert stats.eq(0).all() and weight.eq(0).all()
        d = bo.policy_loss_backward(torch.ones((), device="cuda"), lp, old, adv, weight, mask,
                                    refp, kl_coef=1.0)
        assert d.eq(0).all()
    for shape in ((0, 8), (4, 0), (0, 0)):
        x = torch.zeros(shape, device="cuda")
        stats, weight = bo.policy_loss(x, x, x[:, 0] if shape[1] else x.new_zeros(shape[0]))
        assert stats.eq(0).all() and weight.eq(0).all() and weight.shape == shape[:1]
        assert bo.policy_loss_backward(torch.ones((), device="cuda"), x, x,
                                       x.new_zeros(shape[0]), weight).shape == shape


def test_infinities_that_count():
    """A ratio that overflows: clipped for a positive advantage, infinite loss for a
    negative one; NaN goes through."""
    lp = torch.tensor([[-1.0, -2.0]], device="cuda")
    old = torch.tensor([[-200.0, -2.0]], device="cuda")
    stats, w = bo.policy_loss(lp, old, torch.ones(1, device="cuda"))
    assert abs(stats[0].item() + 1.1) < 1e-6 and stats[3] == 0.5
    stats, _ = bo.policy_loss(lp, old, -torch.ones(1, device="cuda"))
    assert stats[0] == math.inf and stats[3] == 0
    old[0, 1] = math.nan
    stats, _ = bo.policy_loss(lp, old, torch.ones(1, device="cuda"))
    assert stats[0].isnan()
    d = bo.policy_loss_backward(torch.ones((), device="cuda"), lp, old,
                                torch.ones(1, device="cuda"), w)
    assert d[0, 0] == 0 and d[0, 1].isnan()


def test_off_a_boundary():
    args = make(3, 256, True, True, True, 2)

    def shift(t):
        x = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
        return x.copy_(t.view(-1)).view(t.shape)
    stats, d = check(args)
    moved = check(tuple(shift(t) for t in args))
    assert torch.equal(moved[1], d)


def test_captured():
    s = torch.cuda.Stream()
    args = make(6, 300, False, True, True)
    one = torch.ones((), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bo.policy_loss(*args, kl_coef=0.1)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        stats, weight = bo.policy_loss(*args, kl_coef=0.1)
        d = bo.policy_loss_backward(one, *args[:3], weight, *args[3:], kl_coef=0.1)
    for seed in (1, 2):
        for t, v in zip(args, make(6, 300, False, True, True, seed)):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        want, w = bo.policy_loss(*args, kl_coef=0.1)
        assert torch.equal(stats, want) and torch.equal(weight, w)
        assert torch.equal(d, bo.policy_loss_backward(one, *args[:3], w, *args[3:], kl_coef=0.1))
    del g
    bo.release_stream(s)


def test_with_the_cross_entropy():
    """Log probabilities from the vocabulary's cross entropy, and the policy loss's
    gradient back through it, against the same graph in fp64."""
    batch, length, dim, vocab = 4, 70, 64, 500
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(batch, length, dim, device="cuda", generator=g).half().requires_grad_(True)
    w = (0.1 * torch.randn(vocab, dim, device="cuda", generator=g)).half().requires_grad_(True)
    answer = torch.randint(0, vocab, (batch, length), device="cuda", generator=g)
    answer[:, 50:] = -100
    adv = torch.randn(batch, device="cuda", generator=g)
    logp = -nn.linear_cross_entropy(x, w, answer, reduction="none")
    old = (logp + 0.2 * torch.randn(batch, length, device="cuda", generator=g)).detach()
    ref = (logp + 0.3 * torch.randn(batch, length, device="cuda", generator=g)).detach()
    mask = answer != -100
    loss, stats = nn.policy_loss(logp, old, adv, mask, ref, 0.2, 0.3, 0.1, "sequence")
    assert loss.shape == () and not stats.requires_grad and loss.detach() == stats[0]
    grads = torch.autograd.grad(loss * 64, (x, w))
    xd, wd = (t.detach().double().requires_grad_(True) for t in (x, w))
    lp = torch.log_softmax(xd @ wd.T, -1).gather(2, answer.clamp(min=0)[..., None])[..., 0]
    r = torch.exp(lp - old.double())
    a = adv.double()[:, None]
    each = -torch.minimum(r * a, r.clamp(0.8, 1.3) * a)
    e = ref.double() - lp
    each = (each + 0.1 * (torch.expm1(e) - e)) * mask
    want = (each.sum(1) / mask.sum(1)).mean()
    assert abs(loss.item() - want.item()) < 1e-5
    for got, ref_g in zip(grads, torch.autograd.grad(want * 64, (xd, wd))):
        # 16-bit probabilities (2^-11 each, at random) and results
        assert (got.double() - ref_g).norm() <= 2.0 ** -10 * ref_g.norm()


def test_refusals():
    lp, old, adv, mask, refp = make(3, 8, False, True, True)
    with pytest.raises(TypeError):
        bo.policy_loss(lp.half(), old, adv)
    with pytest.raises(TypeError):
        bo.policy_loss(lp, old, adv, mask.float())
    with pytest.raises(ValueError):
        bo.policy_loss(lp, old[:2], adv)
    with pytest.raises(ValueError):
        bo.policy_loss(lp[0], old[0], adv)
    with pytest.raises(ValueError):
        bo.policy_loss(lp, old, adv[:2])
    with pytest.raises(ValueError):
        bo.policy_loss(lp.T, old.T, adv)
    with pytest.raises(ValueError):
        bo.policy_loss(lp, old, adv, reduction="mean")
    with pytest.raises(bo.Fp8OptError):
        bo.policy_loss(lp, old, adv, clip_low=1.5)
    with pytest.raises(ValueError):
        bo.policy_loss_backward(adv, lp, old, adv, adv)


def test_offsets_past_32_bits():
    """2.4e9 tokens, of which the last sequence's last ones differ."""
    batch, length = 3, 800_000_003
    lp = torch.zeros(batch, length, device="cuda")
    old = torch.zeros(batch, length, device="cuda")
    old[2, -3:] = torch.tensor([0.1, -0.1, 1.0], device="cuda")
    adv = torch.tensor([1.0, -2.0, 4.0], device="cuda")
    stats, weight = bo.policy_loss(lp, old, adv)
    # -(1 - 2 + 4) / 3 but for three tokens of 2.4e9; the same number of tokens each
    assert abs(stats[0].item() + 1.0) < 1e-6 and stats[3] == 0
    assert ((weight.double() * (batch * length) - 1).abs() <= 2.0 ** -23).all()
    d = bo.policy_loss_backward(torch.ones((), device="cuda"), lp, old, adv, weight)
    scaled = d[:, -4:].double() * (batch * length)
    want = -adv.double()[:, None] * torch.exp(-old[:, -4:].double())
    assert ((scaled - want).abs() <= 1e-6 * want.abs()).all()
    assert d[0, 0] == -weight[0] and d[1, 0] == 2 * weight[1]
