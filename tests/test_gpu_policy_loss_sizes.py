"""The policy loss of more than 2^32 tokens in vectors of four, with a mask."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_mask_past_2_to_the_32():
    """4.3e9 tokens, of which eleven count, most of them the last ones."""
    import bit_optimizer_gb300 as bo
    batch, length = 3, 1_431_655_772
    assert length % 4 == 0 and batch * length > 2 ** 32
    lp = torch.zeros(batch, length, device="cuda")
    old = torch.zeros(batch, length, device="cuda")
    mask = torch.zeros(batch, length, dtype=torch.bool, device="cuda")
    b = torch.tensor([0, 1] + [2] * 9, device="cuda")
    t = torch.tensor([0, 7] + list(range(length - 9, length)), device="cuda")
    mask[b, t] = True
    old[b, t] = torch.tensor([0.1, -0.05, 0.0, 0.1, -0.1, 1.0, 0.0, 0.02, 0.05, -1.0, 0.15],
                             device="cuda")
    old[2, length - 10] = 5.0                      # masked
    adv = torch.tensor([1.0, -2.0, 4.0], device="cuda")
    stats, weight = bo.policy_loss(lp, old, adv, mask)
    r, a = torch.exp(-old[b, t].double()), adv.double()[b]
    held = r.clamp(0.8, 1.2)
    clipped = held * a < r * a
    each = -torch.minimum(r * a, held * a)
    # a term's exponential, product and place in a sum of nine: 16 roundings
    tol = 16 * 2.0 ** -24 * each.abs().mean()
    assert abs(stats[0].item() - each.mean().item()) <= tol
    assert abs(stats[3].item() - clipped.double().mean().item()) <= 2.0 ** -23
    assert ((weight.double() * 11 - 1).abs() <= 2.0 ** -23).all()
    d = bo.policy_loss_backward(torch.ones((), device="cuda"), lp, old, adv, weight, mask)
    want = torch.where(clipped, 0.0, -r * a) / 11
    assert ((d[b, t].double() - want).abs() <= 8 * 2.0 ** -24 * want.abs()).all()
    d[b, t] = 0
    assert not any(part.any() for part in d.view(-1).split(1 << 28))
    del lp, old, mask, d
    torch.cuda.empty_cache()
