"""The autograd functions against torch's own, and the example that runs the
operators and the optimizer together.

Tolerances.  The 8-bit checkpoints' effect is measured against the same torch
graph on the checkpoint's values, so that only rounding remains: one FP16
rounding (2^-11) of each result and of what went into it, a few of which add up;
16 of them (2^-7) of the 2-norm is allowed.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def near(got, want, tol=2.0 ** -7):
    got, want = got.double(), want.double()
    assert (got - want).norm() <= tol * want.norm() + 1e-12, ((got - want).norm() / want.norm())


def leaves(*shapes, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).half().cuda().requires_grad_(True) for s in shapes]


def test_layer_norm_x_form_matches_torch():
    from bit_optimizer_gb300 import nn
    x, w, b, dy = leaves((3, 50, 96), (96,), (96,), (3, 50, 96))
    y = nn.layer_norm(x, w, b, save="x")
    got = torch.autograd.grad(y, (x, w, b), dy.detach())
    x32, w32, b32 = (t.detach().float().requires_grad_(True) for t in (x, w, b))
    ref = torch.nn.functional.layer_norm(x32, (96,), w32, b32, 1e-5)
    want = torch.autograd.grad(ref, (x32, w32, b32), dy.detach().float())
    near(y, ref)
    for a, r in zip(got, want):
        assert a.dtype == torch.float16
        near(a, r)


def test_fp8_forms_are_the_gradients_at_the_saved_values():
    import bit_optimizer_gb300 as bo
    from bit_optimizer_gb300 import nn
    x, w, b, dy = leaves((200, 128), (64, 128), (64,), (200, 64), seed=1)
    y = nn.linear(x, w, b)
    near(y, torch.nn.functional.linear(x.float(), w.float(), b.float()))
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy.detach())
    saved = bo.act_load(*bo.act_save(x.detach()), torch.float32)
    near(dx, dy.float() @ w.float())
    near(dw, dy.float().T @ saved)
    near(db, dy.float().sum(0))

    g = nn.gelu(x)
    s = saved.requires_grad_(True)
    want = torch.autograd.grad(torch.nn.functional.gelu(s, approximate="tanh"), s,
                               torch.ones_like(s))[0]
    near(g, torch.nn.functional.gelu(x.float(), approximate="tanh"))
    near(torch.autograd.grad(g, x, torch.ones_like(g))[0], want)
    # a gradient that is no contiguous tensor
    expanded = torch.ones(1, 1, device="cuda", dtype=torch.float16).expand(200, 128)
    near(torch.autograd.grad(nn.gelu(x), x, expanded)[0], want)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_linear_cross_entropy_matches_torch(reduction):
    from bit_optimizer_gb300 import nn
    x, w = leaves((4, 40, 64), (1000, 64), seed=2)
    t = torch.randint(0, 1000, (4, 40), generator=torch.Generator().manual_seed(3)).cuda()
    t[:, 30:] = -100
    loss = nn.linear_cross_entropy(x, w, t, reduction=reduction)
    x32, w32 = (a.detach().float().requires_grad_(True) for a in (x, w))
    ref = torch.nn.functional.cross_entropy((x32 @ w32.T).view(-1, 1000), t.view(-1),
                                            reduction=reduction).view(loss.shape)
    near(loss, ref, 1e-5)
    seed = torch.rand(loss.shape, device="cuda") + 0.5
    for a, r in zip(torch.autograd.grad(loss, (x, w), seed),
                    torch.autograd.grad(ref, (x32, w32), seed)):
        near(a, r)


def test_the_mean_over_no_token_is_zero():
    from bit_optimizer_gb300 import nn
    x, w = leaves((8, 64), (100, 64), seed=4)
    t = torch.full((8,), -100, device="cuda")
    loss = nn.linear_cross_entropy(x, w, t)
    assert loss.item() == 0
    assert all((g == 0).all() for g in torch.autograd.grad(loss, (x, w)))


def test_the_example_learns():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_lm
    losses = train_lm.train(steps=60, tokens=2048, vocab=503, dim=128)
    assert abs(losses[0] - 6.22) < 0.5          # log(503): nothing learnt yet
    assert losses[-1] < 0.6 * losses[0]
