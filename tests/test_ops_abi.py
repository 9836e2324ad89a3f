"""The training operators' C entry points refuse malformed calls before any
CUDA call, and the binding refuses CPU tensors."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from bit_optimizer_gb300 import _lib
    return _lib


P = 0x1000   # an address that is never read


def text(lib):
    return lib.load().fp8opt_last_error().decode()


def test_activation_checkpoints(lib):
    L = lib.load()
    assert L.fp8_act_save(P, -1, 0, P, P, None) == lib.ERR_ARG
    assert L.fp8_act_save(P, 2 ** 41, 0, P, P, None) == lib.ERR_ARG
    assert L.fp8_act_save(P, 8, 3, P, P, None) == lib.ERR_UNSUPPORTED
    assert L.fp8_act_save(None, 8, 0, P, P, None) == lib.ERR_ARG
    assert "fp8_act_save" in text(lib) and "NULL" in text(lib)
    assert L.fp8_act_save(P, 8, 0, None, P, None) == lib.ERR_ARG
    assert L.fp8_act_save(P, 8, 0, P, None, None) == lib.ERR_ARG
    assert L.fp8_act_load(P, P, 8, 9, P, None) == lib.ERR_UNSUPPORTED
    assert L.fp8_act_load(P, P, 8, 1, None, None) == lib.ERR_ARG
    assert L.fp8_act_save(None, 0, 0, None, None, None) == lib.OK
    assert L.fp8_act_load(None, None, 0, 0, None, None) == lib.OK
    assert L.fp8_gelu(P, 8, 0, 2, P, P, P, None) == lib.ERR_UNSUPPORTED
    assert "form" in text(lib)
    assert L.fp8_gelu(P, 8, 0, 1, None, P, P, None) == lib.ERR_ARG
    assert L.fp8_gelu_backward(P, P, P, 8, 0, -1, P, None) == lib.ERR_UNSUPPORTED
    assert L.fp8_gelu_backward(P, None, P, 8, 0, 0, P, None) == lib.ERR_ARG
    assert L.fp8_gelu(None, 0, 0, 0, None, None, None, None) == lib.OK


def test_layer_norm(lib):
    L = lib.load()

    def norm(x=P, w=P, b=P, rows=4, cols=8, dt=0, wdt=0, eps=1e-5, y=P, mean=P, rstd=P,
             codes=None, scales=None):
        return L.fp8_layer_norm(x, w, b, rows, cols, dt, wdt, eps, y, mean, rstd, codes, scales,
                                None)
    assert norm(rows=-1) == lib.ERR_ARG and norm(cols=0) == lib.ERR_ARG
    assert norm(rows=2 ** 30, cols=2 ** 30) == lib.ERR_ARG
    assert norm(dt=5) == lib.ERR_UNSUPPORTED and norm(wdt=-1) == lib.ERR_UNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(eps=eps) == lib.ERR_ARG
    assert norm(x=None) == norm(w=None) == norm(y=None) == norm(rstd=None) == lib.ERR_ARG
    assert norm(mean=None) == lib.ERR_ARG                       # neither form
    assert norm(codes=P, scales=P) == lib.ERR_ARG               # both
    assert norm(mean=None, codes=P) == lib.ERR_ARG              # half of one
    assert norm(rows=0, x=None, y=None, mean=None, rstd=None) == lib.OK

    def grad(dy=P, x=P, mean=P, codes=None, scales=None, rstd=P, w=P, rows=4, cols=8, dt=0,
             wdt=0, dx=P, dw=P, db=P):
        return L.fp8_layer_norm_backward(dy, x, mean, codes, scales, rstd, w, rows, cols, dt,
                                         wdt, dx, dw, db, None)
    assert grad(rows=-1) == grad(cols=0) == lib.ERR_ARG
    assert grad(dt=7) == grad(wdt=7) == lib.ERR_UNSUPPORTED
    assert grad(dy=None) == grad(rstd=None) == grad(dx=None) == grad(dw=None) == lib.ERR_ARG
    assert grad(x=None) == grad(mean=None) == grad(x=None, mean=None) == lib.ERR_ARG
    assert grad(codes=P, scales=P) == lib.ERR_ARG
    assert grad(x=None, mean=None, codes=P) == lib.ERR_ARG


def test_linear_cross_entropy(lib):
    L = lib.load()

    def loss(x=P, w=P, t=P, rows=4, dim=8, vocab=16, dt=1, out=P, lse=P):
        return L.fp8_linear_xent(x, w, t, rows, dim, vocab, dt, -100, out, lse, None)
    assert loss(rows=-1) == loss(dim=0) == loss(vocab=0) == lib.ERR_ARG
    assert loss(rows=2 ** 31) == loss(dim=2 ** 31) == loss(vocab=2 ** 31) == lib.ERR_ARG
    assert loss(dt=0) == loss(dt=4) == lib.ERR_UNSUPPORTED
    assert loss(x=None) == loss(w=None) == loss(t=None) == loss(out=None) == lib.ERR_ARG
    assert loss(rows=0, x=None, t=None, out=None, lse=None) == lib.OK

    def grad(dl=P, x=P, w=P, t=P, lse=P, rows=4, dim=8, vocab=16, dt=1, dx=P, dw=P):
        return L.fp8_linear_xent_backward(dl, x, w, t, lse, rows, dim, vocab, dt, -100, dx, dw,
                                          None)
    assert grad(rows=-1) == grad(vocab=0) == lib.ERR_ARG
    assert grad(dt=0) == lib.ERR_UNSUPPORTED
    assert grad(dl=None) == grad(lse=None) == grad(dx=None) == grad(dw=None) == lib.ERR_ARG


def test_linear_cross_entropy_refuses_sums_longer_than_its_tiles_count(lib):
    """dim, and backward the tokens, are summed in blocks of 64 whose number has
    24 bits; the first size past that is refused, the vocabulary is not bound."""
    L = lib.load()
    most = 2 ** 30 - 64
    for dim in (most + 1, 2 ** 30, 2 ** 31 - 1):
        assert L.fp8_linear_xent(P, P, P, 1, dim, 1, 1, -100, P, P, None) == lib.ERR_ARG
        assert L.fp8_linear_xent_backward(P, P, P, P, P, 1, dim, 1, 1, -100, P, P,
                                          None) == lib.ERR_ARG
    assert L.fp8_linear_xent_backward(P, P, P, P, P, most + 1, 1, 1, 1, -100, P, P,
                                      None) == lib.ERR_ARG
    # accepted sizes get as far as the NULL pointer
    assert L.fp8_linear_xent(None, P, P, 2 ** 31 - 1, 1, 2 ** 31 - 1, 1, -100, P, P,
                             None) == lib.ERR_ARG and "NULL" in text(lib)
    assert L.fp8_linear_xent_backward(P, None, P, P, P, most, 1, 1, 1, -100, P, P,
                                      None) == lib.ERR_ARG and "NULL" in text(lib)


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    import bit_optimizer_gb300 as bo
    x, w = torch.zeros(4, 8), torch.zeros(8)
    for call in (lambda: bo.act_save(x), lambda: bo.gelu(x), lambda: bo.layer_norm(x, w, w),
                 lambda: bo.linear_cross_entropy(x.half(), x.half(), torch.zeros(4).long())):
        with pytest.raises(TypeError):
            call()


def test_constants_agree_with_the_header(lib, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "c.c"
    src.write_text('#include <stdio.h>\n#include "fp8opt.h"\nint main(void) { printf("%d %d %d", '
                   'FP8OPT_ACT_GROUP, FP8OPT_GELU_ERF, FP8OPT_GELU_TANH); return 0; }\n')
    exe = tmp_path / "c"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert got.split() == [str(lib.ACT_GROUP), str(lib.GELU_ERF), str(lib.GELU_TANH)]
    assert C.sizeof(C.c_void_p) == 8
