"""The cross entropy at sizes that take its longer paths: several pieces of the
vocabulary backward (a launch holds one piece's dx and dw and the next piece's p;
dx is added to the earlier pieces'), ranges of dx's sum with nothing in them, more
tokens than one forward launch takes.  Every element is compared with float64,
under the tolerances of test_gpu_linear_xent.py.  How many pieces a call took is
read from its launches, so that no change of the rule leaves the path untested.
"""
import pytest
import torch

from test_gpu_linear_xent import check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


def pieces(bo, call):
    """Pieces that a backward call took: its launches but the last."""
    bo.timing_enable(True)
    try:
        call()
        torch.cuda.synchronize()
        return bo.timing_read("xent_grads")[0] - 1
    finally:
        bo.timing_enable(False)


@pytest.mark.parametrize("dtype,rows,dim", [(torch.bfloat16, 8100, 72), (torch.float16, 8192, 65),
                                            (torch.float16, 12001, 264)])
def test_three_pieces_and_more(bo, dtype, rows, dim):
    for vocab in (33003, 66007, 132011):       # odd: the last piece is a short one
        x, w, t, dloss = inputs(rows, dim, vocab, dtype, seed=dim)
        lse = torch.zeros(rows, device="cuda")
        n = pieces(bo, lambda: bo.linear_cross_entropy_backward(dloss, x, w, t, lse))
        if n >= 3:
            break
    assert n >= 3
    # targets at both ends and around every place where a piece can end
    edges = torch.arange(0, vocab, 256, device="cuda")
    t[:len(edges)] = edges
    t[len(edges):2 * len(edges)] = (edges - 1) % vocab
    t[-1] = vocab - 1
    loss, lse = check_forward(bo, x, w, t)
    dx, dw = check_backward(bo, x, w, t, dloss, lse)
    again = bo.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("rows,dim,vocab", [(128, 64, 4300), (1, 64, 4300), (90, 300, 4211)])
def test_ranges_of_the_sum_with_nothing_in_them(bo, rows, dim, vocab):
    """68 blocks of k in 16 ranges: five each, and none for the last two."""
    x, w, t, dloss = inputs(rows, dim, vocab, torch.float16, seed=rows, ignored=0.1)
    check_backward(bo, x, w, t, dloss)


@pytest.mark.parametrize("dim", [24, 17])
def test_more_tokens_than_a_forward_launch_takes(bo, dim):
    x, w, t, dloss = inputs(65536 + 300, dim, 515, torch.bfloat16, seed=dim)
    bo.timing_enable(True)
    try:
        bo.linear_cross_entropy(x, w, t)
        torch.cuda.synchronize()
        assert bo.timing_read("xent_logits")[0] >= 2
    finally:
        bo.timing_enable(False)
    loss, lse = check_forward(bo, x, w, t)
    check_backward(bo, x, w, t, dloss, lse)
