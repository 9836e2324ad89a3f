"""The C entry points of the embedding, the policy loss and distillation refuse malformed calls
before any CUDA call, and the binding refuses CPU tensors."""
import math

import pytest

P = 0x1000   # an address that is never read


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from bit_optimizer_gb300 import _lib
    return _lib


def text(lib):
    return lib.load().fp8opt_last_error().decode()


def test_embedding(lib):
    L = lib.load()

    def lookup(ids=P, w=P, rows=4, dim=8, vocab=16, dt=1, scale=1.0, y=P):
        return L.fp8_embedding(ids, w, rows, dim, vocab, dt, scale, y, None)
    assert lookup(rows=-1) == lookup(dim=0) == lookup(vocab=0) == lib.ERR_ARG
    assert lookup(rows=2 ** 31) == lookup(vocab=2 ** 31) == lib.ERR_ARG
    assert lookup(dim=2 ** 40) == lookup(rows=2 ** 30, dim=2 ** 20) == lib.ERR_ARG
    assert lookup(dt=3) == lookup(dt=-1) == lib.ERR_UNSUPPORTED
    for scale in (math.inf, -math.inf, math.nan):
        assert lookup(scale=scale) == lib.ERR_ARG and "scale" in text(lib)
    assert lookup(ids=None) == lookup(w=None) == lookup(y=None) == lib.ERR_ARG
    assert "fp8_embedding" in text(lib) and "NULL" in text(lib)
    assert lookup(rows=0, ids=None, w=None, y=None) == lib.OK

    def grad(dy=P, ids=P, rows=4, dim=8, vocab=16, dt=1, scale=1.0, pad=-1, dw=P):
        return L.fp8_embedding_backward(dy, ids, rows, dim, vocab, dt, scale, pad, dw, None)
    assert grad(rows=-1) == grad(dim=0) == grad(vocab=0) == grad(vocab=2 ** 31) == lib.ERR_ARG
    assert grad(dt=4) == lib.ERR_UNSUPPORTED
    assert grad(scale=math.nan) == lib.ERR_ARG
    assert grad(dy=None) == grad(ids=None) == grad(dw=None) == lib.ERR_ARG
    assert grad(rows=0, dy=None, ids=None, dw=None) == lib.ERR_ARG


def test_policy_loss(lib):
    L = lib.load()

    def loss(lp=P, old=P, adv=P, mask=P, ref=P, batch=2, length=8, per=0, low=0.2, high=0.2,
             kl=0.1, red=0, stats=P, weight=P):
        return L.fp8_policy_loss(lp, old, adv, mask, ref, batch, length, per, low, high, kl, red,
                                 stats, weight, None)

    def grad(dl=P, lp=P, old=P, adv=P, weight=P, mask=P, ref=P, batch=2, length=8, per=0,
             low=0.2, high=0.2, kl=0.1, d=P):
        return L.fp8_policy_loss_backward(dl, lp, old, adv, weight, mask, ref, batch, length,
                                          per, low, high, kl, d, None)
    for f in (loss, grad):
        assert f(batch=-1) == f(length=-1) == f(batch=2 ** 31) == f(length=2 ** 31) == lib.ERR_ARG
        assert f(batch=2 ** 30, length=2 ** 20) == lib.ERR_ARG
        for low in (-0.1, 1.1, math.nan):
            assert f(low=low) == lib.ERR_ARG and "clip_low" in text(lib)
        for high in (-0.1, math.nan):
            assert f(high=high) == lib.ERR_ARG and "clip_high" in text(lib)
        for kl in (math.inf, math.nan):
            assert f(kl=kl) == lib.ERR_ARG and "kl_coef" in text(lib)
        assert f(lp=None) == f(old=None) == f(adv=None) == f(weight=None) == lib.ERR_ARG
    assert loss(red=2) == loss(red=-1) == lib.ERR_UNSUPPORTED
    assert loss(stats=None) == lib.ERR_ARG
    assert grad(dl=None) == grad(d=None) == lib.ERR_ARG
    assert grad(batch=0, dl=None, d=None) == grad(length=0, lp=None) == lib.OK


def test_distillation(lib):
    L = lib.load()

    def loss(x=P, w=P, ids=P, logits=P, rows=4, dim=8, vocab=16, k=3, dt=1, ldt=0, t=1.0, out=P,
             lse=P):
        return L.fp8_linear_distill(x, w, ids, logits, rows, dim, vocab, k, dt, ldt, t, out, lse,
                                    None)

    def grad(x=P, w=P, ids=P, logits=P, rows=4, dim=8, vocab=16, k=3, dt=1, ldt=0, t=1.0, out=P,
             lse=P, dl=P, dw=P):
        return L.fp8_linear_distill_backward(dl, x, w, ids, logits, lse, rows, dim, vocab, k, dt,
                                             ldt, t, out, dw, None)
    for f in (loss, grad):
        assert f(rows=-1) == f(dim=0) == f(vocab=0) == f(vocab=2 ** 31) == lib.ERR_ARG
        assert f(k=0) == f(k=-1) == f(k=lib.MOST_TEACHER + 1) == lib.ERR_ARG
        assert f(dt=0) == f(dt=3) == f(ldt=3) == f(ldt=-1) == lib.ERR_UNSUPPORTED
        for t in (0.0, -1.0, math.nan, math.inf, 2.0 ** -21, 2.0 ** 21):
            assert f(t=t) == lib.ERR_ARG and "temperature" in text(lib)
        assert f(x=None) == f(w=None) == f(ids=None) == f(logits=None) == lib.ERR_ARG
        assert f(out=None) == f(lse=None) == lib.ERR_ARG and "NULL" in text(lib)
        assert f(dim=2 ** 30) == lib.ERR_ARG
    assert grad(dl=None) == grad(dw=None) == lib.ERR_ARG
    assert grad(rows=2 ** 30) == lib.ERR_ARG
    assert loss(rows=0, x=None, ids=None, out=None) == lib.OK


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    import bit_optimizer_gb300 as bo
    ids, x = torch.zeros(4).long(), torch.zeros(4, 8)
    for call in (lambda: bo.embedding(ids, x), lambda: bo.embedding_backward(x, ids, 16),
                 lambda: bo.policy_loss(x, x, x[:, 0]),
                 lambda: bo.policy_loss_backward(x[0, 0], x, x, x[:, 0], x[:, 0]),
                 lambda: bo.linear_distillation(x.half(), x.half(), ids[:, None], x[:, :1])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        bo.policy_loss(x, x, x[:, 0], reduction="sum")


def test_constants_agree_with_the_header(lib, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "c.c"
    src.write_text('#include <stdio.h>\n#include "fp8opt.h"\nint main(void) { printf("%d %d %d", '
                   'FP8OPT_MEAN_TOKEN, FP8OPT_MEAN_SEQUENCE, FP8OPT_MOST_TEACHER); return 0; }\n')
    exe = tmp_path / "c"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert got.split() == [str(lib.MEAN_TOKEN), str(lib.MEAN_SEQUENCE), str(lib.MOST_TEACHER)]
