"""The embedding, distillation and the policy loss among other calls: one after
another without a wait, on two streams and from two threads at once, captured with
their autograd functions, and a training step through all of them."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def package():
    global bo, nn
    import bit_optimizer_gb300 as bo
    from bit_optimizer_gb300 import nn


def randn(*shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def calls():
    """Calls of each kernel's every way, as functions of nothing."""
    out = []
    for i, (rows, dim, vocab) in enumerate([(40, 64, 500), (700, 129, 3000), (3000, 256, 900),
                                            (9000, 96, 5003), (20000, 24, 70000)]):
        ids = (torch.arange(rows, device="cuda") ** 2 * 7 + i) % vocab
        w, dy = randn(vocab, dim, seed=i), randn(rows, dim, seed=i + 10)
        out.append(lambda ids=ids, w=w: [bo.embedding(ids, w, 2.0)])
        out.append(lambda ids=ids, dy=dy, vocab=vocab: [bo.embedding_backward(dy, ids, vocab)])
    for i, (b, n) in enumerate([(3, 70), (40, 2000), (2000, 60)]):
        lp, old, ref = (randn(b, n, seed=3 * i + k, dtype=torch.float32) for k in range(3))
        adv = randn(b, seed=i, dtype=torch.float32)
        one = torch.ones((), device="cuda")

        def policy(lp=lp, old=old, adv=adv, ref=ref, one=one):
            stats, weight = bo.policy_loss(lp, old, adv, None, ref, kl_coef=0.1)
            return [stats, weight, bo.policy_loss_backward(one, lp, old, adv, weight, None, ref,
                                                           kl_coef=0.1)]
        out.append(policy)
    for i, (rows, dim, vocab, k) in enumerate([(5, 64, 3000, 20), (100, 72, 700, 90),
                                               (600, 128, 5003, 64), (300, 65, 301, 3)]):
        x, w = randn(rows, dim, seed=i), randn(vocab, dim, seed=i + 5, scale=dim ** -0.5)
        ids = (torch.arange(rows * k, device="cuda") ** 2 % vocab).view(rows, k)
        logits, dloss = randn(rows, k, seed=i), torch.rand(rows, device="cuda") + 0.5
        t = ids[:, 0].contiguous()

        def losses(x=x, w=w, ids=ids, logits=logits, dloss=dloss, t=t):
            loss, lse = bo.linear_distillation(x, w, ids, logits, 2.0)
            loss2, lse2 = bo.linear_cross_entropy(x, w, t)
            return [loss, lse, loss2, lse2,
                    *bo.linear_distillation_backward(dloss, x, w, ids, logits, lse, 2.0),
                    *bo.linear_cross_entropy_backward(dloss, x, w, t, lse2)]
        out.append(losses)
    return out


def alone(fs):
    got = []
    for f in fs:
        got.append(f())
        torch.cuda.synchronize()
    return got


def same(got, want):
    return all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_one_after_another():
    fs = calls()
    want = alone(fs)
    assert all(torch.isfinite(o.float()).all() for outs in want for o in outs)
    for repeat in range(20):
        order = torch.randperm(len(fs), generator=torch.Generator().manual_seed(repeat)).tolist()
        got = [fs[i]() for i in order]
        assert same(got, [want[i] for i in order]), repeat


def test_two_streams_at_once():
    fs = calls()
    want = alone(fs)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for repeat in range(5):
        got = [None] * len(fs)
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for i, f in enumerate(fs):
            with torch.cuda.stream(streams[(i + repeat) % 2]):
                got[i] = f()
        torch.cuda.synchronize()
        assert same(got, want)
    for s in streams:
        bo.release_stream(s)


def test_two_threads():
    fs = calls()
    want = alone(fs)
    failed = []

    def work(shift):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for repeat in range(4):
                got = [fs[(i + shift) % len(fs)]() for i in range(len(fs))]
                s.synchronize()
                if not same(got, [want[(i + shift) % len(fs)] for i in range(len(fs))]):
                    failed.append((shift, repeat))
        bo.release_stream(s)
    threads = [threading.Thread(target=work, args=(k * 5,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_a_stream_that_is_given():
    """stream=: the outputs and the work are that stream's."""
    s = torch.cuda.Stream()
    ids = torch.arange(500, device="cuda") % 90
    w, lp = randn(90, 64, seed=1), randn(4, 50, seed=2, dtype=torch.float32)
    x = randn(30, 64, seed=3)
    k, logits = ids[:60].view(30, 2).contiguous(), randn(30, 2, seed=4)
    want = [bo.embedding(ids, w), *bo.policy_loss(lp, lp, lp[:, 0].contiguous()),
            *bo.linear_distillation(x, w, k, logits)]
    torch.cuda.synchronize()
    got = [bo.embedding(ids, w, stream=s),
           *bo.policy_loss(lp, lp, lp[:, 0].contiguous(), stream=s),
           *bo.linear_distillation(x, w, k, logits, stream=s)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(TypeError):
        bo.embedding(ids, w, stream=3)
    bo.release_stream(s)


def step(tokens, answer, ids, logits, old, adv, wte, ln_w, ln_b):
    """One loss through the embedding, a norm, the cross entropy, the policy loss and
    distillation, and its gradients."""
    h = nn.layer_norm(nn.embedding(tokens, wte, 4.0, padding_idx=0), ln_w, ln_b)
    logp = -nn.linear_cross_entropy(h, wte, answer, reduction="none")
    policy, _ = nn.policy_loss(logp, old, adv, answer != -100)
    loss = policy + 0.5 * nn.linear_distillation(h, wte, ids, logits, 2.0)
    return [loss.detach(), *torch.autograd.grad(loss * 64, (wte, ln_w, ln_b))]


def inputs(seed, batch=4, length=60, dim=64, vocab=400, k=12):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def ints(*shape):
        return torch.randint(0, vocab, shape, device="cuda", generator=g)
    tokens, answer = ints(batch, length), ints(batch, length)
    answer[:, -7:] = -100
    ids, logits = ints(batch, length, k), randn(batch, length, k, seed=seed)
    ids[:, -7:] = -1
    old = -6 + 0.3 * randn(batch, length, seed=seed + 1, dtype=torch.float32)
    adv = randn(batch, seed=seed + 2, dtype=torch.float32)
    return [tokens, answer, ids, logits, old, adv]


def parameters(dim=64, vocab=400):
    p = [randn(vocab, dim, seed=1, scale=0.1, dtype=torch.float16),
         1 + randn(dim, seed=2, scale=0.1, dtype=torch.float16),
         randn(dim, seed=3, scale=0.1, dtype=torch.float16)]
    return [t.requires_grad_(True) for t in p]


def test_a_step_through_all_of_them():
    """Against the same graph in torch, in fp64 on the 16-bit values of the layers
    between (8-bit normalised activations and 16-bit gradients: a few percent)."""
    import torch.nn.functional as F
    args, params = inputs(5), parameters()
    got = step(*args, *params)
    tokens, answer, ids, logits, old, adv = args
    wte, ln_w, ln_b = (p.detach().double().requires_grad_(True) for p in params)
    h = F.layer_norm(F.embedding(tokens, wte, padding_idx=0) * 4.0, (64,), ln_w, ln_b)
    z = h @ wte.T
    mask = answer != -100
    logp = -F.cross_entropy(z.view(-1, 400), answer.view(-1), reduction="none").view(mask.shape)
    r = torch.exp(logp - old.double())
    a = adv.double()[:, None]
    policy = (-torch.minimum(r * a, r.clamp(0.8, 1.2) * a) * mask).sum() / mask.sum()
    logq = torch.log_softmax(logits.double() / 2, -1)
    logp2 = torch.log_softmax(z / 2, -1).gather(-1, ids.clamp(min=0))
    each = (logq.exp() * (logq - logp2)).sum(-1) * mask
    loss = policy + 0.5 * each.sum() / mask.sum()
    assert abs(got[0].item() - loss.item()) < 2e-2 * abs(loss.item()) + 1e-3
    for d, ref in zip(got[1:], torch.autograd.grad(loss * 64, (wte, ln_w, ln_b))):
        assert (d.double() - ref).norm() < 0.1 * ref.norm()


def test_a_captured_step():
    """The step and its gradients in a graph: replays on new inputs give an eager
    step's bits.  (No eager graph of the same leaves may live meanwhile: torch would
    order the capturing stream against the one that graph's leaves were used on.)"""
    s = torch.cuda.Stream()
    args, params = inputs(1), parameters()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*args, *params)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step(*args, *params)
    for seed in (2, 3):
        for t, v in zip(args, inputs(seed)):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step(*args, *params)):
            assert torch.equal(a, b)
    del g, out
    bo.release_stream(s)


def test_under_autocast():
    """FP32 weights get FP32 gradients; distillation's product is autocast's type."""
    args, params = inputs(7), [p.detach().float().requires_grad_(True) for p in parameters()]
    tokens, _, ids, logits = args[:4]
    wte = params[0]
    with torch.autocast("cuda", dtype=torch.bfloat16):
        h = nn.embedding(tokens, wte, 4.0)
        loss = nn.linear_distillation(h, wte, ids, logits.float(), 2.0)
    d, = torch.autograd.grad(loss, wte)
    assert h.dtype == d.dtype == torch.float32
    full = wte.detach().double().requires_grad_(True)
    z = (4 * full[tokens]) @ full.T / 2
    logq = torch.log_softmax(logits.double() / 2, -1)
    each = (logq.exp() * (logq - torch.log_softmax(z, -1).gather(-1, ids.clamp(min=0)))).sum(-1)
    live = (ids >= 0).any(-1)
    want = (each * live).sum() / live.sum()
    ref, = torch.autograd.grad(want, full)
    # 16-bit inputs, p - q and results: some 2^-8 each
    assert abs(loss.item() - want.item()) < 1e-2 * want.item()
    assert (d.double() - ref).norm() < 2.0 ** -6 * ref.norm()


def test_one_token_without_a_dimension():
    w = randn(30, 64, seed=1)
    ids = torch.tensor(7, device="cuda")
    y = bo.embedding(ids, w)
    assert torch.equal(y, w[7])
    dw = bo.embedding_backward(y, ids, 30, 2.0)
    assert torch.equal(dw[7], 2 * w[7]) and dw.count_nonzero() == dw[7].count_nonzero()
