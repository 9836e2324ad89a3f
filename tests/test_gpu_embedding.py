"""The embedding and its table's gradient against the definition in 64 bits: every
type, widths in and off 16-byte vectors, token counts on both sides of the two
ways to sort, vocabularies on both sides of a digit, frequent words that span
many chunks, padding and ids outside the vocabulary."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
types = pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16", "f16"])
# half a step of the smallest numbers of a type
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def package():
    global bo, nn
    import bit_optimizer_gb300 as bo
    from bit_optimizer_gb300 import nn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def words(n, vocab, seed):
    """Frequent words first: a third of all tokens is one word."""
    u = torch.rand(n, device="cuda", generator=gen(seed))
    ids = ((vocab + 1.0) ** u - 1.0).long().clamp(0, vocab - 1)
    return torch.where(torch.rand(n, device="cuda", generator=gen(seed + 1)) < 0.3,
                       torch.full_like(ids, min(3, vocab - 1)), ids)


@types
@pytest.mark.parametrize("n,dim,vocab", [(1, 1, 1), (1, 8, 5), (3, 768, 1000), (33, 129, 257),
                                         (257, 7, 9), (64, 4097, 12), (4099, 64, 50257),
                                         (2, 20000, 3)])
def test_lookup(n, dim, vocab, dtype):
    w = torch.randn(vocab, dim, device="cuda", generator=gen(n)).to(dtype)
    ids = words(n, vocab, n)
    for scale in (1.0, math.sqrt(dim), -0.3):
        y = bo.embedding(ids, w, scale)
        assert y.dtype == dtype and y.shape == (n, dim)
        # one product in fp32, one rounding: the same two steps
        assert torch.equal(y, (w[ids].float() * scale).to(dtype))
        exact = w[ids].double() * torch.tensor(scale).double().item()
        assert ((y.double() - exact).abs()
                <= exact.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -23) + TINY[dtype]).all()


def test_lookup_shapes_and_ids_outside_the_vocabulary():
    w = torch.randn(10, 16, device="cuda").half()
    ids = torch.tensor([[0, 9, 10], [-1, -100, 2 ** 40]], device="cuda")
    y = bo.embedding(ids, w)
    assert y.shape == (2, 3, 16)
    assert torch.equal(y[0, 0], w[0]) and torch.equal(y[0, 1], w[9])
    assert y[0, 2].isnan().all() and y[1].isnan().all()
    odd = bo.embedding(ids, w[:, :15].contiguous())
    assert torch.equal(odd[0, :2], w[[0, 9], :15]) and odd[1].isnan().all()
    assert bo.embedding(ids[:0], w).shape == (0, 3, 16)
    assert bo.embedding(ids[0, 0], w).shape == (16,)
    # infinities and NaN of the table go through
    w[0, 0], w[0, 1] = math.inf, math.nan
    y = bo.embedding(torch.zeros(1, dtype=torch.long, device="cuda"), w, 2.0)
    assert y[0, 0] == math.inf and y[0, 1].isnan() and y[0, 2] == 2 * w[0, 2]


def reference(dy, ids, vocab, scale, padding):
    """The gradient in fp64, and the sum of absolute values and the count that its
    fp32 sums' error goes by."""
    keep = (ids >= 0) & (ids < vocab)
    if padding is not None:
        keep &= ids != padding
    at, d = ids[keep], dy[keep].double()
    out = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out).index_add_(0, at, d.abs()) * abs(scale)
    out.index_add_(0, at, d)
    count = torch.bincount(at, minlength=vocab)[:, None]
    return out * scale, size, count


def check(dw, dy, ids, vocab, scale=1.0, padding=None):
    ref, size, count = reference(dy, ids, vocab, scale, padding)
    assert dw.dtype == dy.dtype and dw.shape == ref.shape
    # n - 1 sums and a product in fp32, each off by 2^-24 of at most the absolute
    # sum, the scale's own rounding, and one rounding to the type
    bound = (ref.abs() * torch.finfo(dy.dtype).eps / 2 + (count + 2) * 2.0 ** -24 * size * 1.01
             + TINY[dy.dtype])
    bound[count[:, 0] == 0] = 0.0
    assert ((dw.double() - ref).abs() <= bound).all()


SIZES = [(1, 8, 5), (2, 64, 1), (31, 129, 257), (32, 256, 2), (33, 1024, 3), (64, 7, 255),
         (65, 2056, 256), (1000, 1, 257), (2049, 96, 65535), (8192, 24, 65536), (8193, 40, 65537),
         (20000, 264, 50257), (70001, 33, 300), (70001, 8, 2 ** 24 + 3), (300000, 16, 1000)]


@types
@pytest.mark.parametrize("n,dim,vocab", SIZES)
def test_gradient(n, dim, vocab, dtype):
    if vocab > 2 ** 24 and dtype != torch.float16:
        pytest.skip("one type of the largest vocabulary")
    ids = words(n, vocab, n + dim)
    dy = torch.randn(n, dim, device="cuda", generator=gen(n)).to(dtype)
    dw = bo.embedding_backward(dy, ids, vocab)
    check(dw, dy, ids, vocab)
    assert torch.equal(dw, bo.embedding_backward(dy, ids, vocab))


@pytest.mark.parametrize("n,dim,vocab", SIZES)
def test_whole_numbers_add_up_exactly(n, dim, vocab):
    """Sums of small whole numbers are exact in fp32: every token is in its word's
    sum once, and in no other."""
    ids = words(n, vocab, n)
    dy = torch.randint(-8, 9, (n, dim), device="cuda", generator=gen(1)).float()
    ref = torch.zeros(vocab, dim, device="cuda").index_add_(0, ids, dy)
    assert torch.equal(bo.embedding_backward(dy, ids, vocab), ref)


@pytest.mark.parametrize("n", [31, 32, 64, 65, 4097, 8192, 8200, 40000])
@pytest.mark.parametrize("dim", [8, 515, 1030])
def test_one_word(n, dim):
    """All tokens one word: its sum spans every chunk."""
    dy = torch.randint(-8, 9, (n, dim), device="cuda", generator=gen(n)).float()
    for word, vocab in ((0, 1), (4, 7)):
        ids = torch.full((n,), word, device="cuda")
        dw = bo.embedding_backward(dy, ids, vocab)
        assert torch.equal(dw[word], dy.sum(0))
        assert dw.count_nonzero() == dw[word].count_nonzero()


@pytest.mark.parametrize("n", [40, 5000, 9000])
def test_words_that_start_and_end_at_chunks(n):
    """Runs of 1 to 100 tokens in order, reversed and shuffled: starts and ends at
    every place of a chunk."""
    runs = torch.randint(1, 101, (n // 30 + 2,), generator=torch.Generator().manual_seed(n))
    ids = torch.repeat_interleave(torch.arange(len(runs)) * 3, runs)[:n].cuda()
    vocab = 3 * len(runs)
    dy = torch.randint(-8, 9, (len(ids), 48), device="cuda", generator=gen(n)).float()
    for order in (torch.arange(len(ids)), torch.arange(len(ids)).flip(0),
                  torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))):
        i = ids[order.cuda()]
        ref = torch.zeros(vocab, 48, device="cuda").index_add_(0, i, dy)
        assert torch.equal(bo.embedding_backward(dy, i, vocab), ref)


@types
@pytest.mark.parametrize("n,dim,vocab", [(50, 17, 40), (700, 64, 33), (9001, 64, 500)])
def test_scale_padding_and_ids_outside_the_vocabulary(n, dim, vocab, dtype):
    ids = words(n, vocab, n)
    ids[::7] = vocab - 1
    ids[1::11] = -100
    ids[2::13] = vocab
    ids[3::17] = 2 ** 33 + 1
    dy = torch.randn(n, dim, device="cuda", generator=gen(n)).to(dtype)
    dy[ids == vocab - 1] = math.nan          # padding takes no part whatever it holds
    dy[(ids < 0) | (ids >= vocab)] = math.inf
    dw = bo.embedding_backward(dy, ids, vocab, 2.5, vocab - 1)
    assert dw[vocab - 1].count_nonzero() == 0
    check(dw, dy, ids, vocab, 2.5, vocab - 1)
    # without padding_idx the word is one like the others
    dy[ids == vocab - 1] = 1.0
    check(bo.embedding_backward(dy, ids, vocab, -0.5), dy, ids, vocab, -0.5)


def test_nothing_left():
    dy = torch.randn(300, 24, device="cuda").half()
    for n in (0, 5, 300):
        ids = torch.full((n,), -100, device="cuda")
        assert bo.embedding_backward(dy[:n], ids, 11).eq(0).all()
        assert bo.embedding_backward(dy[:n], ids + 103, 11, padding_idx=3).eq(0).all()
    ids = torch.full((9000,), -1, device="cuda")
    dw = bo.embedding_backward(torch.ones(9000, 24, device="cuda"), ids, 11)
    assert dw.eq(0).all()


def test_offsets_past_32_bits():
    """A table of 2.3e9 elements and as many of tokens."""
    vocab, dim = 70000, 32784
    w = torch.zeros(vocab, dim, dtype=torch.float16, device="cuda")
    ids = torch.tensor([69999, 65537, 0], device="cuda")
    w[ids] = torch.randn(3, dim, device="cuda", generator=gen(0)).half()
    assert torch.equal(bo.embedding(ids, w), w[ids])
    dw = bo.embedding_backward(w[ids].contiguous(), ids, vocab)
    assert torch.equal(dw, w)
    del dw
    n = torch.arange(vocab, device="cuda")
    y = bo.embedding(n, w)
    assert torch.equal(y, w)
    dw = bo.embedding_backward(y, n % 2, 2)
    even = w[0].float() + (w[69998].float())
    odd = w[69999].float() + w[65537].float()
    assert (dw[0].float() - even).abs().max() <= 2.0 ** -10 * even.abs().max()
    assert (dw[1].float() - odd).abs().max() <= 2.0 ** -10 * odd.abs().max()


def test_views_off_a_boundary():
    """Tensors that start one element behind a 16-byte boundary."""
    n, dim, vocab = 100, 64, 50
    for dtype in TYPES:
        w = torch.randn(vocab * dim + 1, device="cuda").to(dtype)[1:].view(vocab, dim)
        dy = torch.randn(n * dim + 1, device="cuda").to(dtype)[1:].view(n, dim)
        ids = words(n, vocab, 5)
        assert torch.equal(bo.embedding(ids, w), w[ids])
        check(bo.embedding_backward(dy, ids, vocab), dy, ids, vocab)


def test_captured_and_on_another_stream():
    n, dim, vocab = 9000, 128, 700
    dy = torch.randn(n, dim, device="cuda").half()
    s = torch.cuda.Stream()
    few = words(500, vocab, 9)
    ids = words(n, vocab, 8)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bo.embedding_backward(dy, ids, vocab)        # the stream's scratch
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dw = bo.embedding_backward(dy, ids, vocab)
        small = bo.embedding_backward(dy[:500], few, vocab)
        y = bo.embedding(ids, dw)
    for seed in (1, 2):
        ids.copy_(words(n, vocab, seed))
        few.copy_(words(500, vocab, seed + 5))
        g.replay()
        torch.cuda.synchronize()
        check(dw, dy, ids, vocab)
        check(small, dy[:500], few, vocab)
        assert torch.equal(y, dw[ids])
    del g
    bo.release_stream(s)


def test_autograd():
    vocab, dim = 300, 64
    w = torch.randn(vocab, dim, device="cuda").half().requires_grad_(True)
    ids = words(600, vocab, 3).view(3, 200)
    up = torch.randn(3, 200, dim, device="cuda").half()
    y = nn.embedding(ids.T, w, 2.0, padding_idx=5)      # (not contiguous)
    assert torch.equal(y, (w.detach()[ids.T].float() * 2).half())
    g, = torch.autograd.grad(y, w, up.transpose(0, 1))
    check(g, up.reshape(-1, dim), ids.reshape(-1), vocab, 2.0, 5)
    for pad in (-1, vocab):
        with pytest.raises(ValueError):
            nn.embedding(ids, w, padding_idx=pad)


def test_refusals():
    w = torch.randn(10, 8, device="cuda")
    ids = torch.zeros(4, dtype=torch.long, device="cuda")
    with pytest.raises(TypeError):
        bo.embedding(ids.int(), w)
    with pytest.raises(TypeError):
        bo.embedding(ids, w.double())
    with pytest.raises(ValueError):
        bo.embedding(ids, w[0])
    with pytest.raises(ValueError):
        bo.embedding(ids, w.T)
    with pytest.raises(TypeError):
        bo.embedding(ids, w, "big")
    with pytest.raises(bo.Fp8OptError):
        bo.embedding(ids, w, math.inf)
    dy = torch.randn(4, 8, device="cuda")
    with pytest.raises(ValueError):
        bo.embedding_backward(dy, ids[:3], 10)
    with pytest.raises(ValueError):
        bo.embedding_backward(dy, ids, 0)
    for pad in (-1, 10):
        with pytest.raises(ValueError):
            bo.embedding_backward(dy, ids, 10, padding_idx=pad)
    with pytest.raises(ValueError):
        bo.embedding_backward(dy.T, ids, 10)
