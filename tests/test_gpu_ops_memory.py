"""The training operators' scratch where device memory is short."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


def loss_gradient(bo, rows, dim, vocab):
    """A call whose p alone takes 512 bytes a token for up to 256 words."""
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    a, b = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    return lambda **kw: bo.linear_cross_entropy_backward(a, x, w, t, b, **kw)


def test_a_call_whose_scratch_does_not_fit_leaves_no_error_behind(bo):
    """More scratch than any device of this kind has is refused; the next call
    is not, though its launch asks for the last error."""
    total = torch.cuda.mem_get_info()[1]
    x = torch.randn(64, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    y = bo.layer_norm(x, w, w)[0]
    with pytest.raises(bo.Fp8OptError, match="MemoryAllocation"):
        loss_gradient(bo, total // 512 + 1, 1, 1)()
    assert torch.equal(bo.layer_norm(x, w, w)[0], y)
    torch.cuda.synchronize()
