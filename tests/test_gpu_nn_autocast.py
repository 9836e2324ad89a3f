"""The autograd functions under torch.autocast, with FP32 parameters.

Tolerances: one rounding to the 16-bit type (unit roundoff h: 2^-11 fp16, 2^-8
bf16) of each input, result and intermediate, a few of which add up; 16 h of the
2-norm is allowed.  The weight's gradient of ``linear`` is compared at the values
that its 8-bit checkpoint holds.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def leaves(*shapes, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).cuda().requires_grad_(True) for s in shapes]


@pytest.mark.parametrize("inside", [False, True])     # where backward runs
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_linear(dtype, inside):
    import bit_optimizer_gb300 as bo
    from bit_optimizer_gb300 import nn

    def near(got, want):
        got, want = got.double(), want.double()
        assert (got - want).norm() <= 16 * HALF[dtype] * want.norm()
    x, w, b, dy = leaves((200, 128), (64, 128), (64,), (200, 64), seed=1)
    with torch.autocast("cuda", dtype=dtype):
        y = nn.linear(x, w, b)
        if inside:
            grads = torch.autograd.grad(y, (x, w, b), dy.detach().to(dtype))
    if not inside:
        grads = torch.autograd.grad(y, (x, w, b), dy.detach().to(dtype))
    assert y.dtype == dtype and all(g.dtype == torch.float32 for g in grads)
    saved = bo.act_load(*bo.act_save(x.detach().to(dtype)), torch.float32)
    near(y, torch.nn.functional.linear(x, w, b))
    for got, want in zip(grads, (dy @ w, dy.T @ saved, dy.sum(0))):
        near(got, want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_block_and_its_loss(dtype):
    """Norm, linear, GELU, linear and the loss, as a model under autocast calls
    them: FP32 gradients for FP32 parameters, near torch's at the same types (the
    8-bit activations put a few percent on them)."""
    from bit_optimizer_gb300 import nn
    from torch.nn import functional as F
    x, lw, lb, fc, fb, out, wte = leaves((300, 64), (64,), (64,), (256, 64), (256,), (64, 256),
                                         (700, 64), seed=2)
    params = (x, lw, lb, fc, fb, out, wte)
    t = torch.arange(300, device="cuda") * 2
    t[::7] = -100

    def model(norm, linear, gelu, loss):
        h = norm(x, lw, lb)
        h = x + linear(gelu(linear(h, fc * 0.1, fb)), out * 0.1)
        return loss(h, wte * 0.1, t)
    with torch.autocast("cuda", dtype=dtype):
        ours = model(nn.layer_norm, nn.linear, nn.gelu, nn.linear_cross_entropy)
    ref = model(lambda x, w, b: F.layer_norm(x, (64,), w, b), F.linear,
                lambda h: F.gelu(h, approximate="tanh"),
                lambda h, w, t: F.cross_entropy(F.linear(h, w), t))
    assert abs(ours.item() - ref.item()) < 16 * HALF[dtype] * ref.item()
    for a, r in zip(torch.autograd.grad(ours, params), torch.autograd.grad(ref, params)):
        assert a.dtype == torch.float32
        assert (a - r).norm() < 0.1 * r.norm()
