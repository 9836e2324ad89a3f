"""linear_distillation of few tokens takes the logits of their entries from the same
product as the sum of exponentials, as it does for many."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


# rows * k up to 4096, and above
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 256), (24, 32), (16, 256), (128, 32), (65, 63),
                                    (33, 125), (100, 64), (128, 256)])
@pytest.mark.parametrize("t", [0.05, 0.5, 1.0])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_token_among_few_and_among_many(bo, rows, k, t, dtype):
    """A student near its teacher, whose loss is small beside its logits.

    Tolerance, derived beforehand: the logits are the same products of 64 terms, so
    the two calls differ in the steps behind them alone: each log sum is off by 2^-18
    and 6 u of the mean of |d| under p, d = (z - max z) / t, and a term q (log q - (d - log
    sum)) by q ((2 |a| + 10) u (|log q - log p| + 1) + 4 u (|log q| + |d| + log sum)), where a
    is the argument of q's exponential."""
    g = torch.Generator().manual_seed(rows)
    many, dim, vocab = 300, 64, 5000
    x = torch.randn(many, dim, generator=g).to(dtype).cuda()
    w = (0.4 * torch.randn(vocab, dim, generator=g)).to(dtype).cuda()
    x[:, 0], w[:, 0] = 4, 5
    t = float(torch.tensor(t).float())
    z = x.double() @ w.double().T
    zk, ids = torch.topk(z, k, 1)
    logits = (zk + 0.1 * t * torch.randn(many, k, generator=g).double().cuda()).float()
    order = torch.randperm(k, generator=g).cuda()
    ids, logits, zk = (a[:, order].contiguous() for a in (ids, logits, zk))
    a, all_lse = bo.linear_distillation(x, w, ids, logits, t)
    b, lse = bo.linear_distillation(x[:rows].contiguous(), w,
                                    ids[:rows].contiguous(), logits[:rows].contiguous(), t)
    d, dk = ((v - z.amax(1, keepdim=True)) / t for v in (z, zk))
    log_sum = torch.logsumexp(d, 1, keepdim=True)
    y = logits.double() / t
    logq = torch.log_softmax(y, 1)
    arg = (y - y.amax(1, keepdim=True)).abs()
    each = torch.exp(logq) * ((2 * arg + 10) * U * ((logq - dk + log_sum).abs() + 1)
                              + 4 * U * (logq.abs() + dk.abs() + log_sum))
    tol = 2.0 ** -18 + 6 * U * (torch.exp(d - log_sum) * d.abs()).sum(1) + each.sum(1)
    assert ((a[:rows] - b).double().abs() <= 2 * tol[:rows]).all(), (
        ((a[:rows] - b).double().abs() / tol[:rows]).max())
    assert ((all_lse[:rows] - lse).double().abs()
            <= 2 * tol[:rows] + 2 * U * lse.double().abs()).all()


def test_entries_of_few_tokens(bo):
    """A word several times, words at the ends of the vocabulary and of tiles, ids that
    are not given and ids outside, and tokens without any."""
    g = torch.Generator().manual_seed(2)
    for rows, vocab in ((40, 1027), (128, 257), (5, 32), (33, 1)):
        k = 20
        x = (torch.randint(-8, 9, (rows, 64), generator=g) / 8).half().cuda()
        w = (torch.randint(-8, 9, (vocab, 64), generator=g) / 8).half().cuda()
        ids = torch.randint(0, vocab, (rows, k), generator=g).cuda()
        ids[:, :7] = torch.tensor([0, vocab - 1, 31, 32, 255, 256, 1023], device="cuda") % vocab
        ids[::3, 8:12] = ids[::3, 7:8]
        ids[1::4, 5:9] = -1
        ids[2] = -2 ** 62
        logits = torch.randn(rows, k, generator=g).cuda()
        logits[1, 3] = -math.inf
        y = torch.where(ids >= 0, logits.double(), -math.inf)
        logq = torch.log_softmax(y, 1)
        logp = torch.log_softmax(x.double() @ w.double().T, 1).gather(1, ids.clamp(min=0))
        q = torch.nan_to_num(torch.exp(logq))
        want = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
        loss, _ = bo.linear_distillation(x, w, ids, logits)
        # |log q|, |log p| below 40, some 30 steps
        assert ((loss.double() - want).abs() <= 40 * 30 * U + 2.0 ** -18).all()
        assert loss[2] == 0
        ids[3, 19], ids[4, 0] = vocab, 2 ** 62
        loss, _ = bo.linear_distillation(x, w, ids, logits)
        bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
        bad[3:5] = True
        assert loss[bad].isnan().all()
        assert ((loss.double() - want).abs()[~bad] <= 40 * 30 * U + 2.0 ** -18).all()


def test_odd_rows_and_captured(bo):
    """Rows that TMA cannot read, and new inputs at every replay."""
    g = torch.Generator().manual_seed(3)
    for dim in (65, 64):
        x = torch.randn(24, dim, generator=g).half().cuda()
        w = (0.2 * torch.randn(3000, dim, generator=g)).half().cuda()
        ids = torch.randint(0, 3000, (24, 50), generator=g).cuda()
        logits = torch.randn(24, 50, generator=g).cuda()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            bo.linear_distillation(x, w, ids, logits, 2.0)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = bo.linear_distillation(x, w, ids, logits, 2.0)
        for seed in range(3):
            g2 = torch.Generator().manual_seed(seed)
            ids.copy_(torch.randint(-500, 3000, (24, 50), generator=g2))
            x.copy_(torch.randn(24, dim, generator=g2).half())
            graph.replay()
            torch.cuda.synchronize()
            want = bo.linear_distillation(x, w, ids, logits, 2.0)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        del graph
        bo.release_stream(s)


@pytest.mark.parametrize("rows,k", [(16, 256), (128, 32), (127, 32)])
def test_all_entries_among_few_words(bo, rows, k):
    """The most entries that are not sorted, all of them words of one tile, or one word."""
    g = torch.Generator().manual_seed(rows)
    vocab = 40000
    x = (torch.randint(-8, 9, (rows, 64), generator=g) / 8).half().cuda()
    w = (torch.randint(-8, 9, (vocab, 64), generator=g) / 8).half().cuda()
    logits = torch.randn(rows, k, generator=g).cuda()
    logp = torch.log_softmax(x.double() @ w.double().T, 1)
    logq = torch.log_softmax(logits.double(), 1)
    for first, words in ((0, 128), (19456 + 128, 128), (39999, 1), (777, 1), (39900, 100)):
        ids = (first + torch.randint(0, words, (rows, k), generator=g)).cuda()
        want = (torch.exp(logq) * (logq - logp.gather(1, ids))).sum(1)
        loss, _ = bo.linear_distillation(x, w, ids, logits)
        assert ((loss.double() - want).abs() <= 40 * 30 * U + 2.0 ** -18).all()
