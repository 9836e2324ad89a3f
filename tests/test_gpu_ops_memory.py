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


def room(bytes_left):
    """A tensor that leaves this much of the device's free memory."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return torch.empty(torch.cuda.mem_get_info()[0] - bytes_left, dtype=torch.uint8,
                       device="cuda")


# 2^21 tokens x 8 x 256 words, one piece: p 1 GiB, dx in fp32 (128 columns) 1 GiB, a
# copy of x 32 MiB: 2.03 GiB, and a quarter more 2.54.
ROWS, NEED = 1 << 21, (2 << 30) + (32 << 20)


def test_scratch_without_room_to_grow_takes_what_it_needs(bo):
    call = loss_gradient(bo, ROWS, 8, 256)
    bo.release()
    hog = room(NEED + (300 << 20))       # (the outputs' 34 MB come first)
    dx, dw = call()
    torch.cuda.synchronize()
    assert (dx == 0).all() and (dw == 0).all()
    del hog
    torch.cuda.empty_cache()
    bo.release()


def test_scratch_takes_the_memory_that_torch_caches(bo):
    """As an allocation of torch's own would."""
    call = loss_gradient(bo, ROWS, 8, 256)
    bo.release()
    hog = room(1 << 30)
    del hog                              # torch keeps it, free
    assert torch.cuda.mem_get_info()[0] < NEED
    dx, dw = call()
    torch.cuda.synchronize()
    assert (dx == 0).all() and (dw == 0).all()
    bo.release()
