"""The policy loss's mean over sequences where their own means cancel."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [50, 60, 9000])
def test_means_that_cancel(length):
    """Sequences of 1 to 50 tokens, in vectors and off them, in one piece and in
    several, whose ratios are 1: their means are their advantages, +-1000, which add
    up to a half.

    Tolerance, derived beforehand: a sequence's sum is a whole number below 2^16,
    exact; its mean and at most 15 sums of means are off by 2^-44 of their absolute
    values each (two fp32 numbers, 2^-48 a number, a few roundings a step), and the
    result's rounding and the number of sequences' reciprocal by 2^-24 each."""
    import bit_optimizer_gb300 as bo
    batch = 2002
    g = torch.Generator(device="cuda").manual_seed(length)
    lp = -torch.rand(batch, length, device="cuda", generator=g)
    count = torch.randint(1, 51, (batch, 1), device="cuda", generator=g)
    start = (torch.rand(batch, 1, device="cuda", generator=g) * (length - count + 1)).long()
    start = torch.minimum(start, length - count)
    at = torch.arange(length, device="cuda")
    mask = (at >= start) & (at < start + count)
    adv = torch.where(torch.arange(batch, device="cuda") < 1000, 1000.0, -1000.0)
    adv[2000], adv[2001] = -0.5, 0.0
    adv = adv[torch.randperm(batch, device="cuda", generator=g)]
    stats, weight = bo.policy_loss(lp, lp.clone(), adv, mask, None, reduction="sequence")
    want = 0.5 / batch
    assert abs(stats[1].item() - want) <= 16 * 2.0 ** -44 * 1000 + 2 * 2.0 ** -24 * want
    assert stats[0] == stats[1] and stats[2] == 0 and stats[3] == 0
    exact = 1 / (count[:, 0].double() * batch)
    assert ((weight.double() - exact).abs() <= 2.0 ** -24 * exact).all()
