"""Activation checkpoints, GELU and layer norm on the GPU against their
definitions in float64.

Tolerances, derived beforehand; u = 2^-24, h the unit roundoff of the result's
type (2^-24 fp32, 2^-8 bf16, 2^-11 fp16), d half its least spacing.

* Checkpoints: codes and scales exactly (each step is one IEEE operation: a
  division, a product, a rounding to E4M3), read values exactly too (a division,
  a product, a rounding).
* GELU.  erf form: the error-function formula's 0.75e-7 on Phi plus 16 u for its
  evaluation; tanh form: the exponent's rounding, |u(x)| 4 u where it matters
  (c (1 - c) |u| < 0.3), plus 8 u.  Both are below 2e-6 of |x|, then h of the
  result.  The derivative c + x c' adds x c' (below 1.2) with the same relative
  error, and c's 2e-6: 4e-6 |dy|, then h.
* Layer norm.  A row's sum is a tree over at most 8 values a thread and 2^9
  threads, below 24 additions deep: the mean is off by 24 u mean|x|, and xhat by
  e = 26 u (mean|x| + |mean|) rstd + 40 u |xhat| (rstd's own sums, root and
  product).  y: |w| e + 4 u (|xhat w| + |b|), then h.  The long-row kernels add
  at most cols / 1024 terms per thread first: 24 becomes 24 + cols / 1024.
* Its gradient: m1 = mean h and m2 = mean h xhat are off by 48 u mean|h| and
  48 u mean|h xhat| (xhat itself by 4 u when it comes from x and the given mean
  and rstd: 4 u |x - mean| rstd, plus u |mean| rstd for the difference); dx then
  by rstd (48 u (mean|h| + |xhat| mean|h xhat|) + 8 u (|h| + |m1| + |xhat m2|)).
  dweight and dbias: sums over the rows, at most rows / 16 + 64 additions deep.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
H = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
GROUP = 128


@pytest.fixture(scope="module")
def bo():
    import bit_optimizer_gb300
    return bit_optimizer_gb300


def randn(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def shifted(t):
    """The same values one element off any alignment."""
    return torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)


def close(got, ref, tol):
    dt = got.dtype
    tol = tol + H[dt] * (ref.abs() + tol) + LEAST[dt]
    off = (got.double() - ref).abs() - tol
    assert not torch.isnan(got).any()
    assert off.le(0).all(), (off.max().item(), off.argmax().item())


def checkpoint_reference(x):
    """Codes and scales of fp32 arithmetic on the CPU, one operation at a time."""
    flat = x.detach().float().cpu().reshape(-1)
    n = flat.numel()
    rows = torch.cat([flat, flat.new_zeros(-n % GROUP)]).view(-1, GROUP)
    bad = torch.isnan(rows).any(1) | torch.isinf(rows).any(1)
    amax = rows.abs().amax(1)
    scale = torch.tensor(448.0) / amax
    scale = torch.where((amax > 0) & ~bad & torch.isfinite(scale), scale, 1.0)
    v = rows * scale[:, None]
    codes = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(torch.isfinite(rows), codes, torch.tensor(0x7F, dtype=torch.uint8))
    return codes.view(-1)[:n].view(x.shape), scale


def checkpoint_values(codes, scales):
    v = codes.cpu().view(torch.float8_e4m3fn).float().view(-1)
    r = (torch.tensor(1.0) / scales.cpu()).repeat_interleave(GROUP)[:v.numel()]
    return (v * r).view(codes.shape)


SHAPES = [(1,), (127,), (128,), (129,), (3, 43), (7, 1000), (64, 4096), (1, 33, 65)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("aligned", [True, False])
def test_checkpoint_is_exact(bo, shape, dtype, aligned):
    x = randn(*shape, dtype=dtype, seed=len(shape) + shape[-1], scale=3.0)
    x = x if aligned else shifted(x)
    codes, scales = bo.act_save(x)
    ref_codes, ref_scales = checkpoint_reference(x)
    assert codes.shape == x.shape and codes.dtype == torch.uint8
    assert torch.equal(scales.cpu(), ref_scales)
    assert torch.equal(codes.cpu(), ref_codes)
    values = checkpoint_values(codes, scales)
    for out in DTYPES:
        got = bo.act_load(codes, scales, out)
        assert got.dtype == out and torch.equal(got.cpu(), values.to(out))
    loaded = bo.act_load(shifted(codes), scales, torch.float32)
    assert torch.equal(loaded.cpu(), values)


@pytest.mark.parametrize("dtype", DTYPES)
def test_checkpoint_of_special_groups(bo, dtype):
    x = randn(9, GROUP, dtype=dtype, seed=1)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 9] = float("inf")
    x[4, 0] = float("-inf")
    x[5] = torch.finfo(dtype).max
    x[6] = torch.finfo(dtype).tiny
    x[7, 1:] = 0
    for a in (x, shifted(x)):
        codes, scales = bo.act_save(a)
        ref_codes, ref_scales = checkpoint_reference(a)
        assert torch.equal(scales.cpu(), ref_scales) and torch.equal(codes.cpu(), ref_codes)
        back = bo.act_load(codes, scales, torch.float32)
        assert torch.isnan(back[2, 5]) and torch.isnan(back[3, 9]) and (back[1] == 0).all()


def gelu64(x, form):
    if form == "tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return x * 0.5 * torch.erfc(-x / math.sqrt(2))


def gelu_grad64(x, form):
    x = x.detach().requires_grad_(True)
    return torch.autograd.grad(gelu64(x, form).sum(), x)[0]


@pytest.mark.parametrize("form", ["none", "tanh"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1,), (130,), (5, 777), (40, 512)])
def test_gelu_and_its_gradient(bo, shape, dtype, form):
    x = randn(*shape, dtype=dtype, seed=shape[-1], scale=2.5)
    dy = randn(*shape, dtype=dtype, seed=shape[-1] + 1)
    for a, d in ((x, dy), (shifted(x), shifted(dy))):
        y, codes, scales = bo.gelu(a, form)
        x64 = a.double()
        close(y, gelu64(x64, form), 2e-6 * x64.abs())
        ref_codes, ref_scales = checkpoint_reference(a)
        assert torch.equal(codes.cpu(), ref_codes) and torch.equal(scales.cpu(), ref_scales)
        saved = checkpoint_values(codes, scales).double().cuda()
        dx = bo.gelu_backward(d, codes, scales, form)
        close(dx, d.double() * gelu_grad64(saved, form), 4e-6 * d.double().abs())


@pytest.mark.parametrize("form", ["none", "tanh"])
def test_gelu_far_from_zero(bo, form):
    x = torch.tensor([0.0, -0.0, 5.0, -5.0, 9.0, -9.0, 40.0, -40.0, 1e4, -1e4, 3e18, -3e18,
                      float("nan"), float("inf")], device="cuda").repeat_interleave(GROUP)
    y, codes, scales = bo.gelu(x, form)
    fine = torch.isfinite(x)
    close(y[fine], gelu64(x[fine].double(), form), 2e-6 * x[fine].double().abs())
    assert torch.isnan(y[torch.isnan(x)]).all() and (y[torch.isinf(x)] == float("inf")).all()
    dx = bo.gelu_backward(torch.ones_like(x), codes, scales, form)
    saved = checkpoint_values(codes, scales).cuda()
    ok = torch.isfinite(saved)
    want = torch.where(saved[ok].abs() > 12, (saved[ok] > 0).double(),
                       gelu_grad64(saved[ok].double().clamp(-12, 12), form))
    close(dx[ok], want, torch.full_like(want, 4e-6))
    assert torch.isnan(dx[~ok]).all()


def norm64(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    xhat = (x - mean) * rstd
    y = xhat * w.double()
    return xhat, mean[..., 0], rstd[..., 0], y if b is None else y + b.double()


def norm_slack(x, xhat, mean, rstd):
    deep = 26 + x.shape[-1] / 1024
    spread = x.double().abs().mean(-1, keepdim=True) + mean.abs()[..., None]
    return deep * U * spread * rstd[..., None] + 40 * U * xhat.abs()


def check_norm(bo, x, w, b, eps):
    xhat, mean, rstd, ref = norm64(x, w, b, eps)
    e = norm_slack(x, xhat, mean, rstd)
    tol = w.double().abs() * e + 4 * U * ((xhat * w.double()).abs() +
                                          (0 if b is None else b.double().abs()))
    y, m, r = bo.layer_norm(x, w, b, eps)
    close(y, ref, tol)
    deep = 26 + x.shape[-1] / 1024
    assert (m.double() - mean).abs().le(deep * U * x.double().abs().mean(-1) + 1e-40).all()
    rel = 40 * U + e.amax(-1) / math.sqrt(max(1, x.shape[-1]))
    assert ((r.double() - rstd).abs() / rstd).le(rel + 60 * U).all()
    y8, codes, scales, r8 = bo.layer_norm(x, w, b, eps, save="fp8")
    assert torch.equal(y, y8) and torch.equal(r, r8)
    # the codes: half a spacing of E4M3 (2^-4 of the value, 2^-10 below 2^-6)
    s = scales.double()[..., None]
    v = codes.view(torch.float8_e4m3fn).double() / s
    assert (v - xhat).abs().le(torch.maximum(xhat.abs() * 2.0 ** -4, 2.0 ** -10 / s) * (1 + 1e-5)
                               + e).all()
    amax = xhat.abs().amax(-1)
    want = torch.where(amax > 1e-30, 448.0 / amax, torch.ones_like(amax))
    assert ((scales.double() - want).abs() / want).le(60 * U + e.amax(-1) / amax.clamp(min=1e-30)).all() \
        or (amax <= 1e-30).any()
    return m, r, codes, scales


def check_norm_grad(bo, dy, w, r, need_bias=True, **saved):
    if "x" in saved:
        x64 = saved["x"].double()
        xhat = (x64 - saved["mean"].double()[..., None]) * r.double()[..., None]
        e = (4 * U * xhat.abs() +
             U * (x64.abs() + saved["mean"].double().abs()[..., None]) * r.double()[..., None])
    else:
        xhat = saved["codes"].view(torch.float8_e4m3fn).double() / saved["scales"].double()[..., None]
        e = 2 * U * xhat.abs()
    dx, dw, db = bo.layer_norm_backward(dy, w, r, need_bias=need_bias, **saved)
    d, k = dy.double(), r.double()[..., None]
    h = d * w.double()
    m1, m2 = h.mean(-1, keepdim=True), (h * xhat).mean(-1, keepdim=True)
    deep = 48 + dy.shape[-1] / 1024
    a1 = h.abs().mean(-1, keepdim=True)
    a2 = (h.abs() * (xhat.abs() + e / (deep * U))).mean(-1, keepdim=True)
    tol = k * (deep * U * (a1 + xhat.abs() * a2) + e * m2.abs() +
               8 * U * (h.abs() + m1.abs() + (xhat * m2).abs()))
    close(dx, k * (h - m1 - xhat * m2), tol)
    d2, x2, e2 = (t.reshape(-1, dy.shape[-1]) for t in (d, xhat, e))
    n = 64 + d2.shape[0] / 16
    close(dw, (d2 * x2).sum(0), (d2.abs() * (n * U * x2.abs() + e2)).sum(0))
    if need_bias:
        close(db, d2.sum(0), n * U * d2.abs().sum(0))
    else:
        assert db is None
    assert dw.dtype == w.dtype and dx.dtype == dy.dtype
    return dx, dw, db


NORMS = [(1, 1), (1, 8), (5, 63), (33, 96), (40, 256), (17, 500), (130, 512), (9, 1000),
         (700, 1024), (12, 1500), (50, 2048), (3, 4095), (21, 4096), (5, 5000), (4, 8192),
         (3, 8193), (2, 12288)]


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.float32),
                                          (torch.float16, torch.float16),
                                          (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("rows,cols", NORMS)
def test_layer_norm_and_its_gradient(bo, rows, cols, dtype, wdtype):
    x = randn(rows, cols, dtype=dtype, seed=cols) + 0.3
    w = (1 + 0.3 * randn(cols, seed=cols + 1)).to(wdtype)
    b = (0.2 * randn(cols, seed=cols + 2)).to(wdtype)
    dy = randn(rows, cols, dtype=dtype, seed=cols + 3)
    m, r, codes, scales = check_norm(bo, x, w, b, 1e-5)
    check_norm_grad(bo, dy, w, r, x=x, mean=m)
    check_norm_grad(bo, dy, w, r, codes=codes, scales=scales)


@pytest.mark.parametrize("cols", [512, 513, 4096])
def test_layer_norm_unaligned_and_without_bias(bo, cols):
    x = shifted(randn(11, cols, dtype=torch.bfloat16, seed=1))
    w = shifted(1 + 0.1 * randn(cols, seed=2))
    dy = shifted(randn(11, cols, dtype=torch.bfloat16, seed=3))
    m, r, codes, scales = check_norm(bo, x, w, None, 1e-6)
    check_norm_grad(bo, dy, w, r, need_bias=False, x=x, mean=m)
    check_norm_grad(bo, dy, w, r, codes=shifted(codes), scales=scales)


@pytest.mark.parametrize("cols", [383, 384, 764, 767, 768, 1535, 1536, 3070])
def test_layer_norm_gradient_of_unaligned_rows_near_a_shared_memory_limit(bo, cols):
    """Widths whose row sums take almost 48 KB of a CTA's shared memory."""
    x = shifted(randn(40, cols, dtype=torch.bfloat16, seed=1))
    w = 1 + 0.1 * randn(cols, seed=2)
    dy = shifted(randn(40, cols, dtype=torch.bfloat16, seed=3))
    m, r, codes, scales = check_norm(bo, x, w, None, 1e-6)
    check_norm_grad(bo, dy, w, r, x=x, mean=m)
    check_norm_grad(bo, dy, w, r, codes=shifted(codes), scales=scales)


def test_layer_norm_many_rows(bo):
    """More rows than one visit of every CTA, and a row count that is no
    multiple of the rows a CTA takes at a time."""
    x = randn(9973, 264, dtype=torch.float16, seed=4)
    w = (1 + 0.1 * randn(264, seed=5)).half()
    dy = randn(9973, 264, dtype=torch.float16, seed=6)
    m, r, codes, scales = check_norm(bo, x, w, w, 1e-5)
    check_norm_grad(bo, dy, w, r, x=x, mean=m)
    check_norm_grad(bo, dy, w, r, codes=codes, scales=scales)


@pytest.mark.parametrize("rows,cols", [(5001, 129), (2600, 1023), (1300, 1530), (800, 2049),
                                       (400, 4090), (160, 8185), (150, 8191), (7, 3), (3000, 201),
                                       (2500, 353)])
def test_layer_norm_rows_that_start_anywhere(bo, rows, cols):
    """Several rows a thread, at every offset from a 16-byte boundary that the
    width gives, with a NaN row whose neighbours share its end vectors."""
    x = randn(rows, cols, dtype=torch.bfloat16, seed=cols) + 0.3
    w = (1 + 0.3 * randn(cols, seed=1)).half()
    dy = randn(rows, cols, dtype=torch.bfloat16, seed=2)
    m, r, codes, scales = check_norm(bo, x, w, w, 1e-5)
    check_norm_grad(bo, dy, w, r, x=x, mean=m)
    dx, _, _ = check_norm_grad(bo, dy, w, r, codes=codes, scales=scales)
    y = bo.layer_norm(x, w, w, 1e-5)[0]
    for bad in (0, rows // 2, rows - 1):
        x2, dy2 = x.clone(), dy.clone()
        x2[bad], dy2[bad] = float("nan"), float("inf")
        others = torch.arange(rows, device="cuda") != bad
        y2, codes2, scales2, r2 = bo.layer_norm(x2, w, w, 1e-5, save="fp8")
        assert torch.equal(y2[others], y[others]) and torch.isnan(y2[bad]).all()
        assert torch.equal(codes2[others], codes[others])
        dx2 = bo.layer_norm_backward(dy2, w, r2, codes=codes2, scales=scales2)[0]
        assert torch.equal(dx2[others], dx[others])


def test_layer_norm_writes_its_own_rows_only(bo):
    """Outputs inside larger buffers: what lies beside them keeps its bytes."""
    for rows, cols in ((3, 13), (1, 7), (3, 357), (200, 1021)):
        n = rows * cols
        x = randn(rows, cols, dtype=torch.bfloat16, seed=cols)
        w = torch.ones(cols, device="cuda")
        want = bo.layer_norm(x, w, w, save="fp8")
        room = [torch.full((n + 64,), 7, dtype=t, device="cuda")
                for t in (torch.bfloat16, torch.uint8, torch.bfloat16)]
        y, codes, dx = (t[32:32 + n] for t in room)
        scales, r = torch.empty_like(want[2]), torch.empty_like(want[3])
        dw = torch.empty_like(w)
        stream = torch.cuda.current_stream().cuda_stream
        assert bo._lib.load().fp8_layer_norm(
            x.data_ptr(), w.data_ptr(), w.data_ptr(), rows, cols, bo._lib.BF16, bo._lib.F32, 1e-5,
            y.data_ptr(), None, r.data_ptr(), codes.data_ptr(), scales.data_ptr(), stream) == 0
        assert bo._lib.load().fp8_layer_norm_backward(
            x.data_ptr(), None, None, codes.data_ptr(), scales.data_ptr(), r.data_ptr(),
            w.data_ptr(), rows, cols, bo._lib.BF16, bo._lib.F32, dx.data_ptr(), dw.data_ptr(),
            None, stream) == 0
        assert torch.equal(y.view(rows, cols), want[0])
        assert torch.equal(codes.view(rows, cols), want[1])
        back = bo.layer_norm_backward(x, w, r, codes=want[1], scales=want[2], need_bias=False)
        assert torch.equal(dx.view(rows, cols), back[0]) and torch.equal(dw, back[1])
        for t in room:
            assert (t[:32] == 7).all() and (t[32 + n:] == 7).all()


def test_layer_norm_of_special_rows(bo):
    x = randn(7, 640, seed=7)
    x[1] = 2.5                 # constant: variance 0
    x[2] = 0
    x[3, 17] = float("nan")
    x[4, 600] = float("inf")
    x[5] = x[5] * 1e-3 + 1000  # a mean far above the spread
    w = torch.ones(640, device="cuda")
    y, m, r = bo.layer_norm(x, w, w * 0, 1e-5)
    assert (y[1] == 0).all() and (y[2] == 0).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    good = [0, 5, 6]
    xhat, mean, rstd, ref = norm64(x[good], w, None, 1e-5)
    close(y[good], ref, norm_slack(x[good], xhat, mean, rstd))
    y8, codes, scales, r8 = bo.layer_norm(x, w, w * 0, 1e-5, save="fp8")
    assert (codes[1] == 0).all() and scales[1] == 1 and scales[3] == 1
    assert (codes[3] == 0x7F).all()
    # a NaN row reaches its own dx and the sums, and no other row's dx
    dy = randn(7, 640, seed=8)
    dx, dw, db = bo.layer_norm_backward(dy, w, r8, codes=codes, scales=scales)
    assert torch.isnan(dx[3]).all() and torch.isfinite(dx[good]).all()
    assert torch.isnan(dw).all() and torch.isfinite(db).all()


def test_layer_norm_gradient_against_differences(bo):
    """Slopes of the float64 norm along random directions: the central
    difference is off by O(step^2); the kernel's gradients are in fp32, each
    element off by at most 200 u of the largest terms."""
    x, dy = randn(6, 200, seed=9), randn(6, 200, seed=10)
    w, b = 1 + 0.2 * randn(200, seed=11), 0.1 * randn(200, seed=12)
    _, m, r = bo.layer_norm(x, w, b, 1e-5)
    grads = bo.layer_norm_backward(dy, w, r, x=x, mean=m)
    args = [x.double(), w.double(), b.double()]
    step = 1e-5
    for i, grad in enumerate(grads):
        d = randn(*args[i].shape, seed=20 + i).double()

        def f(s):
            a = [t + (s * d if k == i else 0) for k, t in enumerate(args)]
            return (norm64(a[0], a[1], a[2], 1e-5)[3] * dy.double()).sum()
        slope = (f(step) - f(-step)) / (2 * step)
        got = (grad.double() * d).sum()
        tol = 200 * U * (grad.double().abs() * d.abs()).sum() + 1e-7 * slope.abs() + 1e-6
        assert (got - slope).abs() <= tol


def test_gelu_gradient_against_differences(bo):
    x = randn(64, 128, seed=13)
    for form in ("none", "tanh"):
        _, codes, scales = bo.gelu(x, form)
        saved = bo.act_load(codes, scales, torch.float32).double()
        dx = bo.gelu_backward(torch.ones_like(x), codes, scales, form)
        step = 1e-5
        slope = (gelu64(saved + step, form) - gelu64(saved - step, form)) / (2 * step)
        assert (dx.double() - slope).abs().max() < 5e-6


def test_no_rows_and_no_elements(bo):
    w = torch.ones(16, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    y, m, r = bo.layer_norm(x, w, w)
    assert y.shape == (0, 16) and m.shape == r.shape == (0,)
    dx, dw, db = bo.layer_norm_backward(x, w, r, x=x, mean=m)
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    codes, scales = bo.act_save(x)
    assert codes.shape == (0, 16) and scales.numel() == 0
    assert bo.act_load(codes, scales).shape == (0, 16)
    assert bo.gelu(x)[0].shape == (0, 16)
    assert bo.gelu_backward(x, codes, scales).shape == (0, 16)


def test_a_tensor_past_two_to_the_31_elements(bo):
    """Offsets past 32 bits: the last groups of a large tensor."""
    n = (1 << 31) + 3 * GROUP + 5
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(
        generator=torch.Generator(device="cuda").manual_seed(3))
    y, codes, scales = bo.gelu(x, "tanh")
    part = slice(n - 2 * GROUP - 5, n)
    yp, cp, sp = bo.gelu(x[part].clone(), "tanh")
    assert torch.equal(y[part], yp) and torch.equal(codes[part], cp)
    assert torch.equal(scales[-3:], sp)
    dx = bo.gelu_backward(x, codes, scales, "tanh")
    assert torch.equal(dx[part], bo.gelu_backward(x[part].clone(), cp, sp, "tanh"))


def test_same_bits_every_time_and_on_another_stream(bo):
    x, dy = randn(3001, 768, dtype=torch.bfloat16, seed=14), randn(3001, 768, dtype=torch.bfloat16)
    w = torch.ones(768, device="cuda", dtype=torch.float16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = None
    for k in range(4):
        s = side if k % 2 else None
        y, codes, scales, r = bo.layer_norm(x, w, w, save="fp8", stream=s)
        got = [y, codes, scales, r, *bo.layer_norm_backward(dy, w, r, codes=codes, scales=scales,
                                                            stream=s)]
        g, gc, gs = bo.gelu(x, "tanh", stream=s)
        got += [g, gc, gs, bo.gelu_backward(dy, gc, gs, "tanh", stream=s),
                bo.act_load(*bo.act_save(x, stream=s), torch.bfloat16, stream=s)]
        torch.cuda.synchronize()
        first = first or [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_captured_in_a_graph(bo):
    x, w = randn(300, 512, dtype=torch.float16, seed=15), torch.ones(512, device="cuda")
    s = torch.cuda.Stream()

    def step():
        y, codes, scales, r = bo.layer_norm(x, w, w, save="fp8")
        return bo.layer_norm_backward(y, w, r, codes=codes, scales=scales)
    with torch.cuda.stream(s):
        want = step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    # the graph holds the stream's scratch: a call that needs more is refused
    big = randn(9000, 8192, dtype=torch.float16)
    with pytest.raises(bo.Fp8OptError):
        with torch.cuda.stream(s):
            r = torch.ones(9000, device="cuda")
            bo.layer_norm_backward(big, torch.ones(8192, device="cuda"), r, x=big, mean=r)
    del g
    bo.release_stream(s)


def test_refusals(bo):
    x = randn(4, 16, dtype=torch.float16)
    w = torch.ones(16, device="cuda")
    y, m, r = bo.layer_norm(x, w, w)
    codes, scales = bo.act_save(x)
    for call in (lambda: bo.layer_norm(x.cpu(), w, w), lambda: bo.layer_norm(x.double(), w, w),
                 lambda: bo.layer_norm(x, w, w.half()), lambda: bo.layer_norm(x, w.int(), None),
                 lambda: bo.act_save(x.int()), lambda: bo.act_load(codes, scales, torch.int32),
                 lambda: bo.act_load(x, scales), lambda: bo.gelu_backward(x, codes, scales.half()),
                 lambda: bo.layer_norm_backward(x, w, r, x=x.float(), mean=m)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: bo.layer_norm(x.T, w[:4], None), lambda: bo.layer_norm(x, w[:8], None),
                 lambda: bo.layer_norm(x, w, w, save="none"), lambda: bo.gelu(x, "sigmoid"),
                 lambda: bo.gelu(x[:, ::2]), lambda: bo.act_load(codes, scales[:0]),
                 lambda: bo.gelu_backward(x, codes[:2].contiguous(), scales),
                 lambda: bo.layer_norm_backward(x, w, r),
                 lambda: bo.layer_norm_backward(x, w, r, x=x),
                 lambda: bo.layer_norm_backward(x, w, r, x=x, mean=m, codes=codes, scales=r),
                 lambda: bo.layer_norm_backward(x, w, r[:2], x=x, mean=m),
                 lambda: bo.layer_norm(torch.empty(3, 0, device="cuda"), w[:0], None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(bo.Fp8OptError):
        bo.layer_norm(x, w, w, eps=-1.0)
    with pytest.raises(bo.Fp8OptError):
        bo.layer_norm(x, w, w, eps=float("nan"))
