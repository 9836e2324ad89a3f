"""GELU of FP32 tensors, erf form, against the definition in float64.

Tolerances, derived beforehand; u = 2^-24.  Phi below |x| = 1 is 1/2 + x R(x^2):
one rounding of a value below 1 (u / 2), and R's few roundings of x R < 0.35: 3 u
at most; beyond, a tail below 0.16 whose factors carry 2^-22.5 (the exponential),
its fit's 1.1e-7 and ten roundings, 20 u of 0.16, and u / 2 for 1 minus it: 3.2 u.
y = x Phi is then rounded once more.  The gradient adds x phi(x), at most 0.242,
with 3 u from the exponential, x^2 u from its argument (x^2 phi |x| below 0.47) and
3 u for three products: 2.2 u together.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("aligned", [True, False])
def test_values_and_gradients(aligned):
    import bit_optimizer_gb300 as bo
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.linspace(-6, 6, 400001), torch.randn(300000, generator=g),
                   torch.randn(100000, generator=g) * 1e-3]).cuda()
    if not aligned:
        x = torch.cat([x.new_zeros(1), x])[1:]
    y, codes, scales = bo.gelu(x)
    x64 = x.double()
    phi = 0.5 * torch.erfc(-x64 / math.sqrt(2))
    assert ((y.double() - x64 * phi).abs() <= 3.2 * U * x64.abs() + U * (x64 * phi).abs()
            + 2.0 ** -150).all()
    s = bo.act_load(codes, scales, torch.float32).double()
    dx = bo.gelu_backward(torch.ones_like(x), codes, scales)
    want = 0.5 * torch.erfc(-s / math.sqrt(2)) + s * torch.exp(-s * s / 2) / math.sqrt(2 * math.pi)
    assert ((dx.double() - want).abs() <= 5.4 * U + U * want.abs()).all()
