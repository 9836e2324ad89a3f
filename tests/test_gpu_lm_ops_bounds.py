"""Bounds of every write of the embedding, distillation and the policy loss, through
the C entry points, between canary bands (test_gpu_ops_bounds.Call): each way to
sort and to sum, rows in and off 16-byte vectors, tensors at 256-byte boundaries and
one element off them."""
import pytest
import torch
from test_gpu_ops_bounds import TYPES, Call, randn

pytestmark = pytest.mark.gpu
F32, U8 = torch.float32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    import bit_optimizer_gb300 as bo
    return bo.load()


skewed = pytest.mark.parametrize("skewed", [False, True])
types = pytest.mark.parametrize("dt", [0, 1, 2])


def words(rows, vocab):
    """Every third token one word; some outside the vocabulary."""
    ids = torch.arange(rows, device="cuda") * 7 % vocab
    ids[::3] = vocab - 1
    ids[5::17] = vocab
    ids[6::19] = -1
    return ids


@skewed
@types
@pytest.mark.parametrize("rows,dim,vocab", [(1, 1, 1), (3, 8, 2), (40, 13, 70), (256, 64, 33),
                                            (257, 65, 40), (1025, 256, 100), (300, 515, 9),
                                            (4097, 24, 300), (5000, 129, 5)])
def test_embedding(lib, rows, dim, vocab, dt, skewed):
    t, ids = TYPES[dt], words(rows, vocab)
    w = randn(vocab, dim, dtype=t, seed=dim)
    c = Call(skewed)
    c.read(ids), c.read(w), c.write(rows * dim, t)
    c.make(lambda ids, w, y, s: lib.fp8_embedding(ids, w, rows, dim, vocab, dt, 1.5, y, s))
    dy = randn(rows, dim, dtype=t, seed=rows)
    for padding in (-1, vocab - 1):
        c = Call(skewed)
        c.read(dy), c.read(ids), c.write(vocab * dim, t)
        c.make(lambda dy, ids, dw, s: lib.fp8_embedding_backward(
            dy, ids, rows, dim, vocab, dt, 0.5, padding, dw, s))


@skewed
@pytest.mark.parametrize("batch,length", [(1, 1), (3, 7), (2, 128), (5, 1000), (2, 4100), (9, 64),
                                          (300, 33), (1, 9001)])
def test_policy_loss(lib, batch, length, skewed):
    n = batch * length
    lp, old, ref = (randn(n, dtype=F32, seed=k) for k in range(3))
    mask = (randn(n, dtype=F32, seed=4) > -0.5).to(U8)
    dloss, weight = randn(1, dtype=F32, seed=5), randn(batch, dtype=F32, seed=6)
    for per, masked, refd in ((0, True, True), (1, False, False), (1, True, True)):
        adv = randn(n if per else batch, dtype=F32, seed=7)
        inputs = [lp, old, adv, mask, ref]
        keep = [True, True, True, masked, refd]

        def given(p):
            return [a if k else None for a, k in zip(p, keep)]
        c = Call(skewed)
        for t in inputs:
            c.read(t)
        c.write(4, F32), c.write(batch, F32)
        for reduction in (0, 1):
            c.make(lambda *p: lib.fp8_policy_loss(*given(p), batch, length, per, 0.2, 0.3, 0.1,
                                                  reduction, *p[5:]))
        c = Call(skewed)
        for t in (*inputs, dloss, weight):
            c.read(t)
        c.write(n, F32)
        c.make(lambda *p: lib.fp8_policy_loss_backward(
            p[5], *given(p)[:3], p[6], *given(p)[3:], batch, length, per, 0.2, 0.3, 0.1, *p[7:]))


@skewed
@pytest.mark.parametrize("dt,ldt", [(1, 0), (2, 1), (1, 2)])
@pytest.mark.parametrize("rows,dim,vocab,k", [(1, 1, 1, 1), (3, 8, 1, 3), (2, 64, 257, 256),
                                              (33, 7, 50, 33), (70, 64, 301, 70),
                                              (129, 65, 257, 5), (300, 131, 1031, 64),
                                              (257, 200, 513, 129)])
def test_distillation(lib, rows, dim, vocab, k, dt, ldt, skewed):
    t = TYPES[dt]
    x = randn(rows, dim, dtype=t, seed=rows)
    w = randn(vocab, dim, dtype=t, seed=vocab, scale=dim ** -0.5)
    ids = torch.arange(rows * k, device="cuda").view(rows, k) * 11 % vocab
    ids[:, k // 2:][::2] = -1
    logits = randn(rows, k, dtype=TYPES[ldt], seed=3)
    lse = torch.logsumexp(x.float() @ w.float().T, 1)
    dloss = randn(rows, dtype=F32, seed=4)
    c = Call(skewed)
    c.read(x), c.read(w), c.read(ids), c.read(logits), c.write(rows, F32), c.write(rows, F32)
    c.make(lambda x, w, ids, logits, loss, lse, s: lib.fp8_linear_distill(
        x, w, ids, logits, rows, dim, vocab, k, dt, ldt, 1.5, loss, lse, s))
    c = Call(skewed)
    c.read(dloss), c.read(x), c.read(w), c.read(ids), c.read(logits), c.read(lse)
    c.write(rows * dim, t), c.write(vocab * dim, t)
    c.make(lambda dloss, x, w, ids, logits, lse, dx, dw, s: lib.fp8_linear_distill_backward(
        dloss, x, w, ids, logits, lse, rows, dim, vocab, k, dt, ldt, 1.0, dx, dw, s))
