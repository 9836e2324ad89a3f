"""The embedding at the borders between its kernels: 256, 4096 tokens and one more,
chunks of 8, 16 and 32 tokens, and tensors of more than 2^32 elements and vectors.
Sums of small whole numbers are exact in fp32, so values are compared for equality."""
import pytest
import torch
from test_gpu_embedding import TYPES, check, gen, words

pytestmark = pytest.mark.gpu
COUNTS = [255, 256, 257, 300, 1024, 4095, 4096, 4097]


@pytest.fixture(scope="module", autouse=True)
def package():
    global bo
    import test_gpu_embedding
    import bit_optimizer_gb300 as bo
    test_gpu_embedding.bo = bo


def whole(n, dim, seed=1):
    return torch.randint(-8, 9, (n, dim), device="cuda", generator=gen(seed)).float()


def added(dy, ids, vocab):
    return torch.zeros(vocab, dy.shape[1], device="cuda").index_add_(0, ids, dy)


@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("dim,vocab", [(8, 50257), (515, 300), (1030, 7)])
def test_whole_numbers(n, dim, vocab):
    ids, dy = words(n, vocab, n), whole(n, dim)
    assert torch.equal(bo.embedding_backward(dy, ids, vocab), added(dy, ids, vocab))


@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("dim", [8, 515, 1030])
def test_one_word(n, dim):
    dy = whole(n, dim, n)
    for word, vocab in ((0, 1), (4, 7)):
        ids = torch.full((n,), word, device="cuda")
        assert torch.equal(bo.embedding_backward(dy, ids, vocab), added(dy, ids, vocab))


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [256, 257, 4096, 4097])
def test_gradient(n, dtype):
    vocab = 700
    ids = words(n, vocab, n)
    ids[::5], ids[1::9], ids[2::50] = vocab - 1, -1, vocab
    for dim in (264, 77):
        dy = torch.randn(n, dim, device="cuda", generator=gen(n)).to(dtype)
        check(bo.embedding_backward(dy, ids, vocab, 0.3, vocab - 1), dy, ids, vocab, 0.3, vocab - 1)


# Chunks have 32 tokens where there are 16 warps for each of 152 SMs with them, else
# 16 or 8; a warp has 128 columns.
@pytest.mark.parametrize("n,dim", [(300, 48), (1000, 48), (4090, 48),
                                   (4000, 1250), (20000, 256),      # chunks of 16
                                   (4000, 2500), (20000, 512), (20000, 509)])   # of 32
def test_words_that_start_and_end_at_chunks(n, dim):
    runs = torch.randint(1, 101, (n // 30 + 2,), generator=torch.Generator().manual_seed(n))
    ids = torch.repeat_interleave(torch.arange(len(runs)) * 3, runs)[:n].cuda()
    vocab, n = 3 * len(runs), len(ids)
    dy = whole(n, dim, n)
    for order in (torch.arange(n), torch.arange(n).flip(0),
                  torch.randperm(n, generator=torch.Generator().manual_seed(1))):
        i = ids[order.cuda()]
        assert torch.equal(bo.embedding_backward(dy, i, vocab), added(dy, i, vocab))


@pytest.mark.parametrize("dim", [32784, 32785])
def test_table_gradient_past_2_to_the_32_elements(dim):
    """4.4e9 elements; few tokens, the short sort and the long one."""
    vocab = 134000
    for n in (200, 3000, 5000):
        ids = torch.randperm(vocab, device="cuda", generator=gen(n))[:n]
        ids[1:4] = torch.tensor([vocab - 1, 0, 65537], device="cuda")
        ids[::20] = vocab - 2                   # (over several chunks)
        dy = torch.randint(-8, 9, (n, dim), device="cuda", generator=gen(n)).half()
        dw = bo.embedding_backward(dy, ids, vocab)
        unique, at = ids.unique(return_inverse=True)
        assert torch.equal(dw[unique].float(), added(dy.float(), at, len(unique)))
        dw[unique] = 0
        assert not any(part.any() for part in dw.split(8192))
        del dw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dim", [32784, 32785])
def test_tokens_past_2_to_the_32_elements(dim):
    n, vocab = 134000, 11
    ids = torch.arange(n, device="cuda") % 7
    dy = torch.zeros(n, dim, dtype=torch.float16, device="cuda")
    some = torch.tensor([0, 1, 40000, 65536, 131071, 131072, n - 2, n - 1], device="cuda")
    dy[some] = torch.randint(-8, 9, (len(some), dim), device="cuda", generator=gen(1)).half()
    dw = bo.embedding_backward(dy, ids, vocab)
    assert torch.equal(dw.float(), added(dy[some].float(), ids[some], vocab))
    del dy
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dim,dtype", [(4096, torch.float32), (4097, torch.float16)])
def test_lookup_past_2_to_the_32(dim, dtype):
    """2^32 vectors of 16 bytes and some, and as many single elements."""
    n = (2 ** 22 if dim == 4096 else 2 ** 20) + 3
    w = torch.randn(9, dim, device="cuda", generator=gen(dim)).to(dtype)
    ids = torch.randint(0, 9, (n,), device="cuda", generator=gen(2))
    y = bo.embedding(ids, w)
    step = 1 << 17
    for a in range(0, n, step):
        assert torch.equal(y[a:a + step], w[ids[a:a + step]])
    del y
    torch.cuda.empty_cache()
