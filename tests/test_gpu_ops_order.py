"""Calls of the training operators that follow one another on a stream without
a wait between them, each reading what the one before wrote, or taking over its
multiprocessors and scratch: the same bits as the calls one at a time."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


def randn(*shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def test_tensor_core_launches_back_to_back(bo):
    """Launches of one tile and of many, whose pairs of CTAs follow one another
    on the same multiprocessors: the barriers of one launch are the shared
    memory of the next."""
    calls = []
    for i, (rows, dim, vocab) in enumerate([(1, 8, 1), (300, 64, 700), (24, 768, 5003),
                                            (129, 136, 257), (700, 256, 9000)]):
        x = randn(rows, dim, dtype=torch.bfloat16, seed=i)
        w = randn(vocab, dim, dtype=torch.bfloat16, seed=i + 10, scale=dim ** -0.5)
        t = torch.arange(rows, device="cuda") * 7 % vocab
        calls.append((x, w, t, torch.rand(rows, device="cuda") + 0.5))

    def both(x, w, t, dloss):
        loss, lse = bo.linear_cross_entropy(x, w, t)
        return [loss, lse, *bo.linear_cross_entropy_backward(dloss, x, w, t, lse)]
    alone = []
    for c in calls:
        alone.append(both(*c))
        torch.cuda.synchronize()
    assert all(torch.isfinite(o.float()).all() for outs in alone for o in outs)
    for repeat in range(30):
        rows = [both(*c) for c in calls]
        for got, want in zip(rows, alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want)), repeat
