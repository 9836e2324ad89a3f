"""Measured cases of the operators at the two ends of a language model: the
embedding lookup and its gradient, distillation of a linear layer over a large
vocabulary from a teacher's top logits, and the clipped policy loss with a KL
term on the tokens' log probabilities, each with its backward pass.

``run`` takes a prepared state through one pass: with ``own`` false in a plain
form of elementary torch operations in fp32, rounded once at the end (in fp64
where fp32 loses digits: long sums, the border of the clipping, the KL term of
nearly equal probabilities); with ``own`` true through this package's entry
points.  ``exact`` evaluates the definitions in 64 bits.

Model sizes are the ones of this repository's synthetic GPT workloads: hidden
sizes 768, 1024 and 2048, vocabulary 50257.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.04


def listed():
    return [
        # the lookup of one short sequence of a 124M model: latency
        dict(name="emb_fwd_128x768", op="emb_fwd", rows=128, dim=768, vocab=50257,
             dtype="f16", scale=1.0, pad=False),
        # the lookup of a 1.3B model's batch with a ragged token count, rows
        # scaled by the root of the width
        dict(name="emb_fwd_16381x2048", op="emb_fwd", rows=16381, dim=2048,
             vocab=50257, dtype="bf16", scale=math.sqrt(2048), pad=False),
        # the dense gradient of a 124M model's micro-batch
        dict(name="emb_bwd_2047x768", op="emb_bwd", rows=2047, dim=768,
             vocab=50257, dtype="f16", scale=1.0, pad=False),
        # the dense gradient of a 350M model's batch, padded at its end
        dict(name="emb_bwd_65536x1024", op="emb_bwd", rows=65536, dim=1024,
             vocab=50257, dtype="bf16", scale=32.0, pad=True),
        # distilling a few tokens: one pass over the vocabulary's weights
        dict(name="distill_fwd_24x768_k32", op="distill_fwd", rows=24, dim=768,
             vocab=50257, k=32, dtype="f16", tdtype="f32", temperature=1.0),
        # distilling a 350M model's batch with a ragged token count
        dict(name="distill_fwd_8191x1024_k64", op="distill_fwd", rows=8191,
             dim=1024, vocab=50257, k=64, dtype="bf16", tdtype="bf16",
             temperature=2.0),
        # its gradients for a 124M model's micro-batch, more of the teacher
        dict(name="distill_bwd_2048x768_k128", op="distill_bwd", rows=2048,
             dim=768, vocab=50257, k=128, dtype="f16", tdtype="f16",
             temperature=1.0),
        # its gradients for a 1.3B model's batch with a ragged token count
        dict(name="distill_bwd_8191x2048_k64", op="distill_bwd", rows=8191,
             dim=2048, vocab=50257, k=64, dtype="bf16", tdtype="f32",
             temperature=2.0),
        # one group of eight short answers: latency
        dict(name="policy_fwd_8x512", op="policy_fwd", batch=8, length=512,
             per_token=False, ref=True, reduction="token"),
        # a batch of 512 long answers, one mean for each
        dict(name="policy_fwd_512x8192", op="policy_fwd", batch=512, length=8192,
             per_token=False, ref=True, reduction="sequence"),
        # 64 answers of an odd length with an advantage for each token, no
        # reference model
        dict(name="policy_bwd_64x1023", op="policy_bwd", batch=64, length=1023,
             per_token=True, ref=False, reduction="sequence"),
        # the gradient of the batch of long answers
        dict(name="policy_bwd_512x8192", op="policy_bwd", batch=512, length=8192,
             per_token=False, ref=True, reduction="token"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A width between lo and hi: mostly a multiple of `step`, else any."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.25 else max(step, n // step * step)


def draw(rng):
    op = rng.choice(["emb_fwd", "emb_bwd", "distill_fwd", "distill_bwd",
                     "policy_fwd", "policy_bwd"])
    half = rng.choice(["bf16", "f16"])
    if op.startswith("emb"):
        dim = _width(rng, 64, 8192, 64)
        return dict(op=op, rows=_log_int(rng, 1, min(131072, (1 << 26) // dim)),
                    dim=dim, vocab=_log_int(rng, 1000, 50257),
                    dtype="f32" if rng.random() < 0.15 else half,
                    scale=rng.choice([1.0, math.sqrt(dim)]), pad=rng.random() < 0.5)
    if op.startswith("distill"):
        return dict(op=op, rows=_log_int(rng, 1, 8191), dim=_width(rng, 64, 2048, 64),
                    vocab=_log_int(rng, 1000, 50257), k=_log_int(rng, 1, 256),
                    dtype=half, tdtype=rng.choice(["f32", "bf16", "f16"]),
                    temperature=rng.choice([1.0, 2.0, round(rng.uniform(0.5, 4.0), 2)]))
    length = _log_int(rng, 1, 32768)
    batch = _log_int(rng, max(1, 64 // length), min(4096, (1 << 22) // length))
    return dict(op=op, batch=batch, length=length, per_token=rng.random() < 0.5,
                ref=rng.random() < 0.7, reduction=rng.choice(["token", "sequence"]))


# ------------------------------------------------------------------ inputs

def _words(rows, vocab, g):
    """Token ids: frequent words first, as a tokenizer's merges give them."""
    u = torch.rand(rows, device="cuda", generator=g)
    return ((vocab + 1.0) ** u - 1.0).long().clamp_(0, vocab - 1)


def _embedding_state(s, g):
    rows, dim, vocab, dt = s["rows"], s["dim"], s["vocab"], DTYPES[s["dtype"]]
    s["ids"] = _words(rows, vocab, g)
    s["padding_idx"] = None
    if s["pad"]:                      # the last sixteenth of the tokens is padding
        s["padding_idx"] = vocab - 1
        s["ids"][rows - rows // 16:] = vocab - 1
    if s["op"] == "emb_fwd":
        w = torch.randn(vocab, dim, device="cuda", generator=g)
        s["w"] = w.mul_(0.02).to(dt)
    else:
        dy = torch.randn(rows, dim, device="cuda", generator=g)
        s["dy"] = dy.mul_(1e-2).to(dt)
    return s


def _distillation_state(s, g):
    rows, dim, vocab, k = s["rows"], s["dim"], s["vocab"], s["k"]
    dt, t = DTYPES[s["dtype"]], s["temperature"]
    s["x"] = torch.randn(rows, dim, device="cuda", generator=g).to(dt)
    w = torch.randn(vocab, dim, device="cuda", generator=g)
    s["w"] = w.mul_(1.5 / math.sqrt(dim)).to(dt)
    ids, top, lse = [], [], []
    for a in range(0, rows, 2048):
        z = (s["x"][a:a + 2048] @ s["w"].T).float()
        lse.append(torch.logsumexp(z / t, 1))
        # a teacher that agrees with the student in part
        z += 1.5 * torch.randn(z.shape, device="cuda", generator=g)
        z, i = torch.topk(z, k, 1)
        top.append(z.to(DTYPES[s["tdtype"]]))
        ids.append(i)
    s["ids"], s["logits"] = torch.cat(ids), torch.cat(top)
    # the teacher kept the logits that make up 98% of its top ones; fewer for
    # the others, and none for the last sixteenth of the tokens, which is padding
    q = torch.softmax(s["logits"].float(), 1)
    s["ids"][q.cumsum(1) - q > 0.98] = -1
    s["ids"][rows - rows // 16:] = -1
    if s["op"] == "distill_bwd":
        # the gradient of the mean over tokens, times a loss scale
        s["dloss"] = torch.full((rows,), 1024.0 / max(1, rows - rows // 16), device="cuda")
        s["lse"] = torch.cat(lse)
    return s


def _policy_state(s, g):
    b, n = s["batch"], s["length"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)
    s["logp"] = -torch.exp(1.2 * randn(b, n) - 1.0)
    s["old"] = s["logp"] + 0.15 * randn(b, n)          # a few updates ago
    s["refp"] = s["logp"] + 0.3 * randn(b, n) if s["ref"] else None
    s["advantage"] = randn(b, n) if s["per_token"] else randn(b)
    # the prompt first, then the answer, then padding; some answers are empty
    at = torch.arange(n, device="cuda")
    first = (0.3 * n * torch.rand(b, 1, device="cuda", generator=g)).long()
    last = first + ((n + 1 - first) * torch.rand(b, 1, device="cuda", generator=g)).long()
    s["mask"] = (at >= first) & (at < last)
    for name in ("old", "refp"):                       # nothing computed outside the answers
        if s[name] is not None:
            s[name] = torch.where(s["mask"], s[name], torch.full_like(s["logp"], -math.inf))
    if s["op"] == "policy_bwd":
        s["weight"] = _weights(s["mask"], s["reduction"])
        s["dloss"] = torch.rand((), device="cuda", generator=g) + 0.5
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    s = dict(case)
    if s["op"].startswith("emb"):
        return _embedding_state(s, g)
    return (_distillation_state if s["op"].startswith("distill") else _policy_state)(s, g)


# -------------------------------------------------------------- plain forms

def _weights(mask, reduction):
    """What each sequence's tokens weigh in the mean: one over all tokens, or
    one over the sequence's and over the sequences that have any."""
    count = mask.sum(1)
    if reduction == "token":
        w = torch.where(count > 0, 1.0 / count.sum(), 0.0)
    else:
        w = torch.where(count > 0, 1.0 / (count * (count > 0).sum()), 0.0)
    return w.float()


def _policy_parts(s):
    """Per token: ratio, whether it is clipped, KL argument, and advantage."""
    lp, a = s["logp"], s["advantage"]
    a = a if s["per_token"] else a[:, None].expand_as(lp)
    d = lp.double() - s["old"].double()
    clipped = (((a > 0) & (d > math.log1p(CLIP_HIGH)))
               | ((a < 0) & (d < math.log1p(-CLIP_LOW))))
    e = s["refp"].double() - lp.double() if s["ref"] else None
    return torch.exp(lp - s["old"]), clipped, e, a


def _plain_policy(s):
    mask, zero = s["mask"], torch.zeros_like(s["logp"])
    ratio, clipped, e, a = _policy_parts(s)
    if s["op"] == "policy_bwd":
        d = torch.where(clipped, zero, -ratio * a)
        if s["ref"]:
            d = d - KL_COEF * torch.expm1(e).float()
        d = d * (s["dloss"] * s["weight"])[:, None]
        return {"dlogp": torch.where(mask, d, zero)}
    weight = _weights(mask, s["reduction"])
    bound = torch.where(a > 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW)
    policy = -torch.where(clipped, bound * a, ratio * a)
    kl = (torch.expm1(e) - e).float() if s["ref"] else zero
    each = torch.stack([policy, kl, clipped.float()])
    sums = torch.where(mask, each, zero).sum(2, dtype=torch.float64)
    policy, kl, part = (sums * weight).sum(1).unbind()
    return {"stats": torch.stack([policy + KL_COEF * kl, policy, kl, part]).float(),
            "weight": weight}


def _plain_distillation(s):
    x, w, t, ids = s["x"].float(), s["w"].float(), s["temperature"], s["ids"]
    z = x @ w.T / t
    given, at = ids >= 0, ids.clamp(min=0)
    logits = torch.where(given, s["logits"].float() / t, -math.inf)
    live = given.any(1, keepdim=True)
    q = torch.where(live, torch.softmax(logits, 1), 0.0)
    if s["op"] == "distill_fwd":
        top = z.amax(1, keepdim=True)
        lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
        each = q * (torch.log(q) - (z.gather(1, at) - lse))
        loss = torch.where(q > 0, each, 0.0).sum(1)
        return {"loss": loss, "lse": lse[:, 0]}
    p = torch.exp(z - s["lse"][:, None])
    p.scatter_add_(1, at, -q)
    p *= torch.where(live[:, 0], s["dloss"] / t, 0.0)[:, None]
    return {"dx": (p @ w).to(s["x"].dtype), "dw": (p.T @ x).to(s["x"].dtype)}


def _plain_embedding(s):
    if s["op"] == "emb_fwd":
        y = s["w"][s["ids"]].float() * s["scale"]
        return {"y": y.to(s["w"].dtype)}
    dw = torch.zeros(s["vocab"], s["dim"], device="cuda")
    dw.index_add_(0, s["ids"], s["dy"].float())
    if s["padding_idx"] is not None:
        dw[s["padding_idx"]] = 0.0
    return {"dw": (dw * s["scale"]).to(s["dy"].dtype)}


def run(s):
    op = s["op"]
    if not own:
        return (_plain_embedding if op.startswith("emb") else _plain_distillation
                if op.startswith("distill") else _plain_policy)(s)
    import bit_optimizer_gb300 as bo
    if op == "emb_fwd":
        return {"y": bo.embedding(s["ids"], s["w"], s["scale"])}
    if op == "emb_bwd":
        return {"dw": bo.embedding_backward(s["dy"], s["ids"], s["vocab"], s["scale"],
                                            s["padding_idx"])}
    if op == "distill_fwd":
        loss, lse = bo.linear_distillation(s["x"], s["w"], s["ids"], s["logits"],
                                           s["temperature"])
        return {"loss": loss, "lse": lse}
    if op == "distill_bwd":
        dx, dw = bo.linear_distillation_backward(s["dloss"], s["x"], s["w"], s["ids"],
                                                 s["logits"], s["lse"], s["temperature"])
        return {"dx": dx, "dw": dw}
    if op == "policy_fwd":
        stats, weight = bo.policy_loss(s["logp"], s["old"], s["advantage"], s["mask"],
                                       s["refp"], CLIP_LOW, CLIP_HIGH, KL_COEF,
                                       s["reduction"])
        return {"stats": stats, "weight": weight}
    return {"dlogp": bo.policy_loss_backward(s["dloss"], s["logp"], s["old"],
                                             s["advantage"], s["weight"], s["mask"],
                                             s["refp"], CLIP_LOW, CLIP_HIGH, KL_COEF)}


# ------------------------------------------------------------------- work

def _distinct(rows, vocab):
    """How many different words `rows` draws of _words have, on average."""
    v = torch.arange(vocab, dtype=torch.float64)
    p = torch.log((v + 2) / (v + 1)) / math.log(vocab + 1)
    return float((1 - (1 - p) ** rows).sum())


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op.startswith("emb"):
        e, n = size[case["dtype"]], case["rows"] * case["dim"]
        # the rows that are looked up, or all rows of the gradient
        rows = _distinct(case["rows"], case["vocab"]) if op == "emb_fwd" else case["vocab"]
        return {"bytes": e * (n + rows * case["dim"]) + 8 * case["rows"], "flops": n}
    if op.startswith("distill"):
        e, rows, dim, vocab = size[case["dtype"]], case["rows"], case["dim"], case["vocab"]
        teacher = rows * case["k"] * (8 + size[case["tdtype"]])
        forward = op == "distill_fwd"
        # the logits are not kept: one product for them, one for each gradient
        return {"bytes": (1 if forward else 2) * e * dim * (rows + vocab) + teacher + 8 * rows,
                "flops": (2.0 if forward else 6.0) * rows * dim * vocab}
    n, b = case["batch"] * case["length"], case["batch"]
    per = 4 * (2 + case["ref"] + case["per_token"]) + 1
    if op == "policy_bwd":
        per += 4
    return {"bytes": per * n + 4 * b * (2 - case["per_token"]), "flops": 20 * n}


# ------------------------------------------------------------------ exact

def _exact_embedding(s):
    ids, scale = s["ids"], s["scale"]
    if s["op"] == "emb_fwd":
        return {"y": torch.index_select(s["w"], 0, ids).double().mul_(scale)}
    keep = torch.ones_like(ids, dtype=torch.bool)
    if s["padding_idx"] is not None:
        keep = ids != s["padding_idx"]
    # the matrix with a one for each token in its word's row
    where = torch.stack([ids, torch.arange(ids.numel(), device=ids.device)])[:, keep]
    ones = torch.ones(where.shape[1], dtype=torch.float64, device=ids.device)
    m = torch.sparse_coo_tensor(where, ones * scale, (s["vocab"], ids.numel()),
                                check_invariants=False)
    return {"dw": torch.sparse.mm(m, s["dy"].double())}


def _exact_distillation(s):
    w, t = s["w"].double(), s["temperature"]
    dx, dw = torch.zeros_like(s["x"], dtype=torch.float64), torch.zeros_like(w)
    losses, lses = [], []
    for a in range(0, s["rows"], 1024):        # rows of tokens at a time
        x, ids = s["x"][a:a + 1024].double(), s["ids"][a:a + 1024]
        y = s["logits"][a:a + 1024].double() / t
        y = y.masked_fill(ids < 0, -math.inf)
        dead = (ids < 0).all(1)
        y[dead] = 0.0                          # any numbers: they do not count
        logq = y - torch.logsumexp(y, 1, keepdim=True)
        q = torch.exp(logq)
        z = (x @ w.T).div_(t)
        if s["op"] == "distill_fwd":
            logp = z - torch.logsumexp(z, 1, keepdim=True)
            each = torch.where(ids < 0, 0.0, q * (logq - logp.gather(1, ids.clamp(min=0))))
            losses.append(torch.where(dead, 0.0, torch.nansum(each, 1)))
            lses.append(torch.logsumexp(z, 1))
            continue
        r = torch.zeros_like(z).scatter_add_(1, ids.clamp(min=0), torch.where(ids < 0, 0.0, q))
        p = torch.exp(z - s["lse"][a:a + 1024].double()[:, None]).sub_(r)
        p *= (s["dloss"][a:a + 1024].double() / t * ~dead)[:, None]
        dx[a:a + 1024] = p @ w
        dw += p.T @ x
    if s["op"] == "distill_fwd":
        return {"loss": torch.cat(losses), "lse": torch.cat(lses)}
    return {"dx": dx, "dw": dw}


def _exact_policy(s):
    b, n = s["batch"], s["length"]
    m = s["mask"]
    row = torch.arange(b, device=m.device)[:, None].expand(b, n)[m]
    lp, old = s["logp"][m].double(), s["old"][m].double()
    a = (s["advantage"][m] if s["per_token"] else s["advantage"][row]).double()
    r = torch.exp(lp - old)
    low, high = torch.full_like(r, 1 - CLIP_LOW), torch.full_like(r, 1 + CLIP_HIGH)
    held = torch.maximum(torch.minimum(r, high), low)
    clipped = held * a < r * a
    u = torch.exp(s["refp"][m].double() - lp) if s["ref"] else torch.ones_like(r)
    if s["op"] == "policy_bwd":
        g = torch.where(clipped, 0.0, -a * r) + KL_COEF * (1 - u)
        out = torch.zeros(b, n, dtype=torch.float64, device=m.device)
        out[m] = g * s["weight"].double()[row] * s["dloss"].double()
        return {"dlogp": out}
    count = torch.bincount(row, minlength=b).double()
    weight = 1 / count if s["reduction"] == "sequence" else torch.ones_like(count) / len(row)
    weight = torch.where(count > 0, weight, 0.0)
    if s["reduction"] == "sequence":
        weight = weight / (count > 0).sum()
    policy = (torch.maximum(-a * r, -a * held) * weight[row]).sum()
    kl = ((u - 1 - torch.log(u)) * weight[row]).sum()
    part = (clipped.double() * weight[row]).sum()
    return {"stats": torch.stack([policy + KL_COEF * kl, policy, kl, part]), "weight": weight}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("emb"):
        return _exact_embedding(s)
    return (_exact_distillation if s["op"].startswith("distill") else _exact_policy)(s)
