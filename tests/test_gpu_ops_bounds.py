"""Bounds of every write of the training operators, through the C entry points.

Inputs and outputs of a call are carved out of one allocation between bands of 256
bytes, at 256-byte boundaries and one element off them.  After the call every byte
outside the outputs must read as before: the bands, and the inputs.  The call is
made twice over different old contents; the outputs must come out the same, so
each of their bytes was written.  Sizes: single elements, groups and rows that end
within a vector, rows of every form, odd vocabularies and token counts.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
PAD = 256
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}
SIZE = {torch.float32: 4, torch.bfloat16: 2, torch.float16: 2, torch.uint8: 1, torch.int64: 8}


@pytest.fixture(scope="module")
def lib():
    import bit_optimizer_gb300 as bo
    return bo.load()


class Call:
    """Buffers of one call: add them, make(f), then read `out`."""

    def __init__(self, skewed):
        self.skewed, self.parts, self.used = skewed, [], PAD

    def _place(self, n, dtype):
        at = -(-self.used // PAD) * PAD + (SIZE[dtype] if self.skewed else 0)
        self.used = at + n * SIZE[dtype] + PAD
        return at

    def read(self, values):
        self.parts.append((self._place(values.numel(), values.dtype), values, None))
        return len(self.parts) - 1

    def write(self, n, dtype):
        self.parts.append((self._place(n, dtype), None, (n, dtype)))
        return len(self.parts) - 1

    def make(self, f):
        results = []
        for seed in (1, 2):
            g = torch.Generator(device="cuda").manual_seed(seed)
            buf = torch.randint(0, 256, (self.used,), dtype=torch.uint8, device="cuda", generator=g)
            free = torch.zeros(self.used, dtype=torch.bool, device="cuda")
            for at, values, out in self.parts:
                if values is not None:
                    raw = values.reshape(-1).view(torch.uint8)
                    buf[at:at + raw.numel()] = raw
                else:
                    free[at:at + out[0] * SIZE[out[1]]] = True
            before = buf.clone()
            status = f(*(buf.data_ptr() + at for at, _, _ in self.parts),
                       torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert status == 0
            assert torch.equal(buf[~free], before[~free])
            results.append(buf[free])
        assert torch.equal(*results)
        self.out = results[0]


def randn(*shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


skewed = pytest.mark.parametrize("skewed", [False, True])
types = pytest.mark.parametrize("dt", [0, 1, 2])


@skewed
@types
@pytest.mark.parametrize("n", [1, 127, 128, 129, 4096, 70003])
def test_checkpoints_and_gelu(lib, n, dt, skewed):
    t, groups = TYPES[dt], -(-n // 128)
    x = randn(n, dtype=t, seed=n)
    import bit_optimizer_gb300 as bo
    codes, scales = bo.act_save(x)
    c = Call(skewed)
    c.read(x), c.write(n, torch.uint8), c.write(groups, torch.float32)
    c.make(lambda x, codes, scales, s: lib.fp8_act_save(x, n, dt, codes, scales, s))
    c = Call(skewed)
    c.read(codes), c.read(scales), c.write(n, t)
    c.make(lambda codes, scales, x, s: lib.fp8_act_load(codes, scales, n, dt, x, s))
    for form in (0, 1):
        c = Call(skewed)
        c.read(x), c.write(n, t), c.write(n, torch.uint8), c.write(groups, torch.float32)
        c.make(lambda x, y, codes, scales, s: lib.fp8_gelu(x, n, dt, form, y, codes, scales, s))
        c = Call(skewed)
        c.read(x), c.read(codes), c.read(scales), c.write(n, t)
        c.make(lambda dy, codes, scales, dx, s: lib.fp8_gelu_backward(dy, codes, scales, n, dt, form,
                                                                      dx, s))


@skewed
@pytest.mark.parametrize("dt,wdt", [(0, 1), (1, 0), (2, 2)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 13), (70, 63), (17, 256), (5, 357), (1300, 201),
                                       (33, 2041), (3, 2049), (4, 4096), (2, 8191), (2, 8193)])
def test_layer_norm(lib, rows, cols, dt, wdt, skewed):
    t, wt, f32, n = TYPES[dt], TYPES[wdt], torch.float32, rows * cols
    x, dy = randn(n, dtype=t, seed=cols), randn(n, dtype=t, seed=cols + 1)
    w, b = 1 + randn(cols, dtype=wt, seed=1, scale=0.1), randn(cols, dtype=wt, seed=2)
    import bit_optimizer_gb300 as bo
    _, mean, rstd = bo.layer_norm(x.view(rows, cols), w, b)
    _, codes, scales, _ = bo.layer_norm(x.view(rows, cols), w, b, save="fp8")
    c = Call(skewed)
    c.read(x), c.read(w), c.read(b), c.write(n, t), c.write(rows, f32), c.write(rows, f32)
    c.make(lambda x, w, b, y, mean, rstd, s: lib.fp8_layer_norm(
        x, w, b, rows, cols, dt, wdt, 1e-5, y, mean, rstd, None, None, s))
    c = Call(skewed)
    c.read(x), c.read(w), c.write(n, t), c.write(rows, f32)
    c.write(n, torch.uint8), c.write(rows, f32)
    c.make(lambda x, w, y, rstd, codes, scales, s: lib.fp8_layer_norm(
        x, w, None, rows, cols, dt, wdt, 1e-5, y, None, rstd, codes, scales, s))
    c = Call(skewed)
    c.read(dy), c.read(x), c.read(mean), c.read(rstd), c.read(w)
    c.write(n, t), c.write(cols, wt), c.write(cols, wt)
    c.make(lambda dy, x, mean, rstd, w, dx, dw, db, s: lib.fp8_layer_norm_backward(
        dy, x, mean, None, None, rstd, w, rows, cols, dt, wdt, dx, dw, db, s))
    c = Call(skewed)
    c.read(dy), c.read(codes), c.read(scales), c.read(rstd), c.read(w)
    c.write(n, t), c.write(cols, wt)
    c.make(lambda dy, codes, scales, rstd, w, dx, dw, s: lib.fp8_layer_norm_backward(
        dy, None, None, codes, scales, rstd, w, rows, cols, dt, wdt, dx, dw, None, s))


@skewed
@pytest.mark.parametrize("dt", [1, 2])
@pytest.mark.parametrize("rows,dim,vocab", [(1, 1, 1), (3, 8, 1), (2, 64, 257), (33, 7, 50),
                                            (70, 64, 301), (129, 65, 257), (300, 131, 1031),
                                            (257, 200, 513)])
def test_cross_entropy(lib, rows, dim, vocab, dt, skewed):
    t, f32 = TYPES[dt], torch.float32
    x = randn(rows, dim, dtype=t, seed=rows)
    w = randn(vocab, dim, dtype=t, seed=vocab, scale=dim ** -0.5)
    target = torch.arange(rows, device="cuda") * 5 % vocab
    target[rows // 2] = -100
    lse = torch.logsumexp(x.float() @ w.float().T, 1)
    dloss = randn(rows, dtype=f32, seed=3)
    c = Call(skewed)
    c.read(x), c.read(w), c.read(target), c.write(rows, f32), c.write(rows, f32)
    c.make(lambda x, w, target, loss, lse, s: lib.fp8_linear_xent(
        x, w, target, rows, dim, vocab, dt, -100, loss, lse, s))
    c = Call(skewed)
    c.read(dloss), c.read(x), c.read(w), c.read(target), c.read(lse)
    c.write(rows * dim, t), c.write(vocab * dim, t)
    c.make(lambda dloss, x, w, target, lse, dx, dw, s: lib.fp8_linear_xent_backward(
        dloss, x, w, target, lse, rows, dim, vocab, dt, -100, dx, dw, s))
