"""Layer norm in every form of its row accesses (elements, vectors of the flat
tensor, aligned vectors, rows too long for registers) and every type, with more
rows than one visit of every CTA, under the tolerances of test_gpu_ops.py."""
import pytest
import torch

from test_gpu_ops import DTYPES, check_norm, check_norm_grad, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


@pytest.mark.parametrize("dtype,wdtype", [(torch.float32, torch.float32),
                                          (torch.float16, torch.bfloat16),
                                          (torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("rows,cols", [
    (5001, 129), (3000, 201), (2500, 353), (2600, 1023), (1300, 1530), (800, 2049), (400, 4090),
    (160, 8185), (150, 8191),                                        # rows that start anywhere
    (9001, 64), (5003, 768), (1501, 2048), (700, 5120), (320, 8192),    # aligned rows
    (400, 9001)])                                                    # long rows
def test_many_rows(bo, rows, cols, dtype, wdtype):
    x = randn(rows, cols, dtype=dtype, seed=cols) + 0.3
    w = (1 + 0.3 * randn(cols, seed=cols + 1)).to(wdtype)
    b = (0.2 * randn(cols, seed=cols + 2)).to(wdtype)
    dy = randn(rows, cols, dtype=dtype, seed=cols + 3)
    m, r, codes, scales = check_norm(bo, x, w, b, 1e-5)
    check_norm_grad(bo, dy, w, r, x=x, mean=m)
    check_norm_grad(bo, dy, w, r, codes=codes, scales=scales)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_row_is_the_same_wherever_it_lies(bo, dtype):
    """Equal rows of a length that is no multiple of eight, so that they start at
    every offset from a 16-byte boundary: the statistics of all are within a
    rounding or two (the order of the sums goes with the offset), the codes'
    scale with them."""
    row = randn(1, 1021, dtype=dtype, seed=5)
    x = row.expand(2000, 1021).contiguous()
    w = torch.ones(1021, device="cuda")
    _, mean, rstd = bo.layer_norm(x, w, w)
    _, _, scales, _ = bo.layer_norm(x, w, w, save="fp8")
    for t in (mean, rstd, scales):
        assert ((t - t[0]).abs() <= 40 * 2.0 ** -24 * row.float().abs().mean().clamp(min=1)
                * t[0].abs().clamp(min=0.1)).all()
        assert torch.equal(t[::8], t[0].expand(250))      # the same offset: the same bits
