"""Measured cases of the training operators that sit around the FP8 optimizer:
layer norm, 8-bit activation checkpoints (plain and through GELU) and the
softmax cross entropy of a linear layer over a large vocabulary, each with its
backward pass.

``run`` takes a prepared state through one pass: with ``own`` false in a plain
form of elementary torch operations in fp32, rounded once at the end; with
``own`` true through this package's entry points.  FP8 codes come back as
torch.float8_e4m3fn tensors (the code values, one byte each, a view) beside
their fp32 scales.  ``exact`` evaluates the definitions in 64 bits.

Model sizes are the ones of this repository's synthetic GPT workloads: hidden
sizes 768, 1024, 2048 and 4096, feed-forward sizes 4096 to 16384, vocabulary
50257.
"""
import math

import torch

own = False

GROUP = 128        # elements that share one checkpoint scale
FP8_MAX = 448.0    # E4M3
IGNORE = -100      # target of a token that takes no part in the loss
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one short sequence through a 124M model's norm: latency
        dict(name="ln_fwd_128x768", op="ln_fwd", rows=128, cols=768, dtype="f16",
             wdtype="f16", save="x"),
        # a 6.7B model's norm, the input kept as an 8-bit checkpoint
        dict(name="ln_fwd_fp8_16384x4096", op="ln_fwd", rows=16384, cols=4096,
             dtype="bf16", wdtype="f16", save="fp8"),
        # a 350M model's micro-batch, gradient from the 16-bit input
        dict(name="ln_bwd_4096x1024", op="ln_bwd", rows=4096, cols=1024,
             dtype="f16", wdtype="f16", save="x"),
        # a 1.3B model's batch with a ragged token count, gradient from the checkpoint
        dict(name="ln_bwd_fp8_16381x2048", op="ln_bwd", rows=16381, cols=2048,
             dtype="bf16", wdtype="f32", save="fp8"),
        # a checkpoint of an odd-sized activation: 1021 tokens of an odd width
        dict(name="act_save_1021x2049", op="act_save", rows=1021, cols=2049,
             dtype="bf16"),
        # reading a 350M model's feed-forward checkpoint back
        dict(name="act_load_16384x4096", op="act_load", rows=16384, cols=4096,
             dtype="f16"),
        # a 350M model's feed-forward activation in one short sequence
        dict(name="gelu_512x4096", op="gelu_fwd", rows=512, cols=4096,
             dtype="f16", approximate="tanh"),
        # the backward pass of a 6.7B model's feed-forward activation
        dict(name="gelu_bwd_8192x16384", op="gelu_bwd", rows=8192, cols=16384,
             dtype="bf16", approximate="none"),
        # the loss of a few tokens: one pass over the vocabulary's weights
        dict(name="xent_fwd_24x768", op="xent_fwd", rows=24, d=768, vocab=50257,
             dtype="f16"),
        # the loss of a 350M model's batch
        dict(name="xent_fwd_8192x1024", op="xent_fwd", rows=8192, d=1024,
             vocab=50257, dtype="bf16"),
        # the loss gradients of a 124M model's micro-batch
        dict(name="xent_bwd_2048x768", op="xent_bwd", rows=2048, d=768,
             vocab=50257, dtype="f16"),
        # the loss gradients of a 1.3B model's batch with a ragged token count
        dict(name="xent_bwd_8191x2048", op="xent_bwd", rows=8191, d=2048,
             vocab=50257, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A width between lo and hi: mostly a multiple of `step`, else any."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.25 else max(step, n // step * step)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "act_save", "act_load", "gelu_fwd",
                     "gelu_bwd", "xent_fwd", "xent_bwd"])
    half = rng.choice(["bf16", "f16"])
    if op.startswith("xent"):
        d = _width(rng, 64, 2048, 64)
        vocab = _log_int(rng, 1000, 50257)
        return dict(op=op, rows=_log_int(rng, 1, 8191), d=d, vocab=vocab,
                    dtype=half)
    cols = _width(rng, 64, 8192, 64)
    rows = _log_int(rng, 1, min(32768, (1 << 26) // cols))
    dtype = "f32" if rng.random() < 0.15 else half
    if op.startswith("ln"):
        return dict(op=op, rows=rows, cols=cols, dtype=dtype,
                    wdtype=rng.choice(["f32", "bf16", "f16"]),
                    save=rng.choice(["x", "fp8"]))
    if op.startswith("gelu"):
        return dict(op=op, rows=rows, cols=cols, dtype=dtype,
                    approximate=rng.choice(["none", "tanh"]))
    return dict(op=op, rows=rows, cols=cols, dtype=dtype)


# ------------------------------------------------------------------ inputs

def _activation(rows, cols, g):
    """Tokens by channels: unit spread, small channel offsets, and a few
    channels that are far larger than the rest, as transformer activations
    have them."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    gain = torch.exp(0.3 * torch.randn(cols, device="cuda", generator=g))
    big = torch.rand(cols, device="cuda", generator=g) < 0.005
    gain = torch.where(big, gain * 12, gain)
    shift = 0.2 * torch.randn(cols, device="cuda", generator=g)
    return x.mul_(gain).add_(shift)


def _groups(flat):
    """A flat tensor as rows of GROUP elements, zeros after its end."""
    pad = -flat.numel() % GROUP
    return torch.nn.functional.pad(flat, (0, pad)).view(-1, GROUP)


def _encode(v):
    """Rows of fp32 values -> E4M3 codes and one scale a row."""
    amax = v.abs().amax(1)
    scale = torch.where(amax > 0, FP8_MAX / amax, torch.ones_like(amax))
    scale = torch.where(torch.isfinite(scale), scale, torch.ones_like(scale))
    return (v * scale[:, None]).to(torch.float8_e4m3fn), scale


def _decode(codes, scales):
    """E4M3 codes (rows) and their scales -> fp32 values."""
    return codes.view(torch.float8_e4m3fn).float() * (1.0 / scales)[:, None]


def _save(x):
    """A checkpoint: codes in the shape of x, one scale per GROUP elements."""
    codes, scales = _encode(_groups(x.float().view(-1)))
    codes = codes.view(torch.uint8).view(-1)[:x.numel()].contiguous()
    return codes.view(x.shape), scales


def _load(codes, scales):
    v = _decode(_groups(codes.view(-1)).contiguous(), scales)
    return v.view(-1)[:codes.numel()].view(codes.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    op, rows, dt = case["op"], case["rows"], DTYPES[case["dtype"]]
    s = dict(case)
    if op.startswith("xent"):
        d, vocab = case["d"], case["vocab"]
        s["x"] = torch.randn(rows, d, device="cuda", generator=g).to(dt)
        w = torch.randn(vocab, d, device="cuda", generator=g)
        s["w"] = w.mul_(1.5 / math.sqrt(d)).to(dt)
        # frequent tokens first, as a tokenizer's merges give them; the last
        # sixteenth of the tokens is padding
        u = torch.rand(rows, device="cuda", generator=g)
        t = ((vocab + 1.0) ** u - 1.0).long().clamp_(0, vocab - 1)
        t[rows - rows // 16:] = IGNORE
        s["target"] = t
        if op == "xent_bwd":
            # the gradient of the mean over tokens, times a loss scale
            count = max(1, rows - rows // 16)
            s["dloss"] = torch.full((rows,), 1024.0 / count, device="cuda")
            lse = torch.empty(rows, device="cuda")
            for a in range(0, rows, 2048):
                z = s["x"][a:a + 2048].float() @ s["w"].float().T
                lse[a:a + 2048] = torch.logsumexp(z, 1)
            s["lse"] = lse
        return s
    cols = case["cols"]
    x = _activation(rows, cols, g).to(dt)
    if op.startswith("ln"):
        wt = DTYPES[case["wdtype"]]
        s["weight"] = (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(wt)
        s["bias"] = (0.1 * torch.randn(cols, device="cuda", generator=g)).to(wt)
        s["eps"] = 1e-5
        if op == "ln_fwd":
            s["x"] = x
            return s
        s["dy"] = (1e-2 * torch.randn(rows, cols, device="cuda", generator=g)).to(dt)
        x32 = x.float()
        mean = x32.mean(1)
        rstd = 1.0 / torch.sqrt(x32.sub_(mean[:, None]).square().mean(1) + s["eps"])
        s["rstd"] = rstd
        if case["save"] == "x":
            s["x"], s["mean"] = x, mean
        else:
            codes, s["scales"] = _encode(x32.mul_(rstd[:, None]))
            s["codes"] = codes.view(torch.uint8)
        return s
    if op in ("act_save", "gelu_fwd"):
        s["x"] = x
        return s
    s["codes"], s["scales"] = _save(x)
    if op == "gelu_bwd":
        s["dy"] = (1e-2 * torch.randn(rows, cols, device="cuda", generator=g)).to(dt)
    return s


# -------------------------------------------------------------- plain forms

_K0, _K1 = math.sqrt(2 / math.pi), 0.044715


def _plain_gelu(x, approximate):
    if approximate == "tanh":
        return 0.5 * x * (1 + torch.tanh(_K0 * (x + _K1 * x * x * x)))
    return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))


def _plain_gelu_grad(x, approximate):
    if approximate == "tanh":
        t = torch.tanh(_K0 * (x + _K1 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * _K0 * (1 + 3 * _K1 * x * x)
    phi = torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * phi


def _plain(s):
    op, dt = s["op"], DTYPES[s["dtype"]]
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1.0 / torch.sqrt(c.square().mean(1) + s["eps"])
        xhat = c * rstd[:, None]
        y = (xhat * s["weight"].float() + s["bias"].float()).to(dt)
        if s["save"] == "x":
            return {"y": y, "mean": mean, "rstd": rstd}
        codes, scales = _encode(xhat)
        return {"y": y, "codes": codes, "scales": scales, "rstd": rstd}
    if op == "ln_bwd":
        dy, w, rstd = s["dy"].float(), s["weight"].float(), s["rstd"][:, None]
        xhat = ((s["x"].float() - s["mean"][:, None]) * rstd if s["save"] == "x"
                else _decode(s["codes"], s["scales"]))
        wdy = dy * w
        dx = rstd * (wdy - wdy.mean(1, keepdim=True)
                     - xhat * (wdy * xhat).mean(1, keepdim=True))
        wt = s["weight"].dtype
        return {"dx": dx.to(dt), "dweight": (dy * xhat).sum(0).to(wt),
                "dbias": dy.sum(0).to(wt)}
    if op == "act_save":
        codes, scales = _save(s["x"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "act_load":
        return {"x": _load(s["codes"], s["scales"]).to(dt)}
    if op == "gelu_fwd":
        codes, scales = _save(s["x"])
        y = _plain_gelu(s["x"].float(), s["approximate"]).to(dt)
        return {"y": y, "codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "gelu_bwd":
        x = _load(s["codes"], s["scales"])
        return {"dx": (s["dy"].float() * _plain_gelu_grad(x, s["approximate"])).to(dt)}
    x, w, target = s["x"].float(), s["w"].float(), s["target"]
    z = x @ w.T
    keep = target != IGNORE
    at = target.clamp(min=0)[:, None]
    if op == "xent_fwd":
        top = z.amax(1, keepdim=True)
        lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
        loss = torch.where(keep, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
        return {"loss": loss, "lse": lse}
    p = torch.exp(z - s["lse"][:, None])
    p.scatter_add_(1, at, torch.full_like(s["lse"], -1.0)[:, None])
    p *= torch.where(keep, s["dloss"], torch.zeros_like(s["lse"]))[:, None]
    return {"dx": (p @ w).to(dt), "dw": (p.T @ x).to(dt)}


def run(s):
    if not own:
        return _plain(s)
    import bit_optimizer_gb300 as bo
    op = s["op"]
    if op == "ln_fwd":
        if s["save"] == "x":
            y, mean, rstd = bo.layer_norm(s["x"], s["weight"], s["bias"], s["eps"])
            return {"y": y, "mean": mean, "rstd": rstd}
        y, codes, scales, rstd = bo.layer_norm(s["x"], s["weight"], s["bias"],
                                               s["eps"], save="fp8")
        return {"y": y, "codes": codes.view(torch.float8_e4m3fn),
                "scales": scales, "rstd": rstd}
    if op == "ln_bwd":
        if s["save"] == "x":
            dx, dw, db = bo.layer_norm_backward(s["dy"], s["weight"], s["rstd"],
                                                x=s["x"], mean=s["mean"])
        else:
            dx, dw, db = bo.layer_norm_backward(s["dy"], s["weight"], s["rstd"],
                                                codes=s["codes"], scales=s["scales"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "act_save":
        codes, scales = bo.act_save(s["x"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "act_load":
        return {"x": bo.act_load(s["codes"], s["scales"], DTYPES[s["dtype"]])}
    if op == "gelu_fwd":
        y, codes, scales = bo.gelu(s["x"], s["approximate"])
        return {"y": y, "codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "gelu_bwd":
        return {"dx": bo.gelu_backward(s["dy"], s["codes"], s["scales"],
                                       s["approximate"])}
    if op == "xent_fwd":
        loss, lse = bo.linear_cross_entropy(s["x"], s["w"], s["target"], IGNORE)
        return {"loss": loss, "lse": lse}
    dx, dw = bo.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"],
                                              s["target"], s["lse"], IGNORE)
    return {"dx": dx, "dw": dw}


# ------------------------------------------------------------------- work

def work(case):
    op, rows = case["op"], case["rows"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    e = size[case["dtype"]]
    if op.startswith("xent"):
        d, vocab = case["d"], case["vocab"]
        products = 2.0 * rows * d * vocab
        if op == "xent_fwd":
            return {"bytes": e * d * (rows + vocab) + 16 * rows, "flops": products}
        # the logits are not kept: one product for them, one for each gradient
        return {"bytes": 2 * e * d * (rows + vocab) + 16 * rows,
                "flops": 3 * products}
    n = rows * case["cols"]
    scales = 4 * -(-n // GROUP)
    if op.startswith("ln"):
        fp8 = case["save"] == "fp8"
        wb = 2 * size[case["wdtype"]] * case["cols"]
        if op == "ln_fwd":
            return {"bytes": 2 * e * n + (n if fp8 else 0) + 8 * rows + wb,
                    "flops": 8 * n}
        return {"bytes": (2 * e + (1 if fp8 else e)) * n + 8 * rows + 1.5 * wb,
                "flops": 14 * n}
    per = {"act_save": e + 1, "act_load": e + 1, "gelu_fwd": 2 * e + 1,
           "gelu_bwd": 2 * e + 1}[op]
    return {"bytes": per * n + scales,
            "flops": {"act_save": 3, "act_load": 1, "gelu_fwd": 14,
                      "gelu_bwd": 22}[op] * n}


# ------------------------------------------------------------------ exact

def _e4m3_64(v):
    """The E4M3 value nearest to each float64 (ties to even, saturating)."""
    _, e = torch.frexp(v)                       # |v| = f * 2^e, f in [1/2, 1)
    q = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return (torch.round(v / q) * q).clamp(-FP8_MAX, FP8_MAX)


def _codes_64(v):
    """Values of the codes of float64 rows and the rows' scales."""
    amax = v.abs().amax(1, keepdim=True)
    scale = torch.where(amax > 0, FP8_MAX / amax, torch.ones_like(amax))
    return _e4m3_64(v * scale), scale[:, 0]


def _values_64(codes):
    """The values of E4M3 code bytes: sign, 4 exponent bits, 3 fraction bits."""
    b = torch.arange(256, device=codes.device, dtype=torch.float64)
    sign = 1 - 2 * torch.floor(b / 128)
    e, f = torch.floor(b / 8) % 16, b % 8
    v = torch.where(e > 0, (8 + f) * torch.exp2(e - 10), f * torch.exp2(b * 0 - 9))
    return (sign * v)[codes.long()]


def _checkpoint_64(s):
    n = s["codes"].numel()
    r = (1.0 / s["scales"].double()).repeat_interleave(GROUP)[:n]
    return _values_64(s["codes"]) * r.view(s["codes"].shape)


def _saved_64(x):
    flat = x.double().view(-1)
    rows = torch.zeros(-(-flat.numel() // GROUP) * GROUP, dtype=torch.float64,
                       device=x.device)
    rows[:flat.numel()] = flat
    v, scale = _codes_64(rows.view(-1, GROUP))
    return v.view(-1)[:flat.numel()].view(x.shape), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + s["eps"]) ** -0.5
        xhat = (x - mean[:, None]) * rstd[:, None]
        y = torch.addcmul(s["bias"].double(), xhat, s["weight"].double())
        if s["save"] == "x":
            return {"y": y, "mean": mean, "rstd": rstd}
        v, scale = _codes_64(xhat)
        return {"y": y, "codes": v, "scales": scale, "rstd": rstd}
    if op == "ln_bwd":
        dy, w, rstd = s["dy"].double(), s["weight"].double(), s["rstd"].double()
        if s["save"] == "x":
            xhat = (s["x"].double() - s["mean"].double()[:, None]) * rstd[:, None]
        else:
            xhat = _values_64(s["codes"]) / s["scales"].double()[:, None]
        h = dy * w
        a = h.sum(1) / h.shape[1]
        b = torch.einsum("rc,rc->r", h, xhat) / h.shape[1]
        dx = (h - a[:, None] - xhat * b[:, None]) * rstd[:, None]
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xhat),
                "dbias": dy.sum(0)}
    if op == "act_save":
        v, scale = _saved_64(s["x"])
        return {"codes": v, "scales": scale}
    if op == "act_load":
        return {"x": _checkpoint_64(s)}
    if op.startswith("gelu"):
        x = (s["x"].double() if op == "gelu_fwd" else _checkpoint_64(s))
        if s["approximate"] == "tanh":
            u = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
            c = torch.sigmoid(u)
            dc = c * torch.sigmoid(-u) * 2 * math.sqrt(2 / math.pi) * (
                1 + 3 * 0.044715 * x ** 2)
        else:
            c = 0.5 * torch.erfc(-x / math.sqrt(2))
            dc = torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        if op == "gelu_bwd":
            return {"dx": s["dy"].double() * (c + x * dc)}
        v, scale = _saved_64(s["x"])
        return {"y": x * c, "codes": v, "scales": scale}
    w, target = s["w"].double(), s["target"]
    rows = target.numel()
    out = {"loss": torch.zeros(rows, dtype=torch.float64, device=w.device)}
    out["lse"] = torch.zeros_like(out["loss"])
    dx, dw = torch.zeros_like(s["x"], dtype=torch.float64), torch.zeros_like(w)
    for a in range(0, rows, 1024):           # rows of tokens at a time
        x, t = s["x"][a:a + 1024].double(), target[a:a + 1024]
        live = (t != IGNORE).nonzero()[:, 0]
        z = x @ w.T
        if op == "xent_fwd":
            lse = torch.logsumexp(z, 1)
            out["lse"][a:a + 1024] = lse
            out["loss"][a + live] = lse[live] - z[live, t[live]]
            continue
        p = torch.exp(z[live] - s["lse"][a + live].double()[:, None])
        p[torch.arange(live.numel(), device=p.device), t[live]] -= 1
        p *= s["dloss"][a + live].double()[:, None]
        dx[a + live] = p @ w
        dw += p.T @ x[live]
    return out if op == "xent_fwd" else {"dx": dx, "dw": dw}
