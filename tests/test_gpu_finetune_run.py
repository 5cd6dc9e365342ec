"""The fine-tuning calls together, as a training step uses them (B200 only):
a packed batch through one layer of attention to logits, a loss on those, and
the gradients back to every weight, against automatic differentiation of the
same step in 64 bits; and the calls' behaviour at scale, on two captured
graphs at once and when a device wait runs out.

Tolerance of the whole step, in the 2-norm of each gradient relative to its
own: a rounding to bf16 is off by at most 2^-8 of each value.  A gradient
passes through at most ten of them (q|k|v, P, o, its projection, the logits,
their gradient, two products' results, dS, dq|dk|dv), and dS = P (dP - D) is
a difference whose terms may be twice its size, so 2 * 10 * 2^-8 = 0.08.
A log-probability is off by some 0.02 (ten roundings of values near one, of
random sign), a ratio by as much of itself; the preference margin, BETA = 0.02
times a difference of sums over up to 300 positions, by 0.02 * 0.02 * 18, far
less, and the loss by no more than its margin.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

BOUND = 20 * 2.0 ** -8
BETA = 0.02


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def setup(torch, lens, pad, H, Hkv, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()

    d, n, total = 256, sum(lens) + pad, sum(lens)
    w = dict(qkv=randn(d, (H + 2 * Hkv) * 128, scale=d ** -0.5), out=randn(H * 128, d, scale=(H * 128) ** -0.5),
             head=randn(d, V, scale=d ** -0.5))
    x = randn(n, d)
    y = torch.randint(0, V, (n,), generator=g, device="cuda").to(torch.int32)
    y[torch.rand(n, generator=g, device="cuda") < 0.3] = -1   # prompts
    y[total:] = -1
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    extra = dict(adv=torch.randn(n, generator=g, device="cuda"), weight=torch.rand(n, generator=g, device="cuda") / n,
                 ratio=0.1 * torch.randn(n, generator=g, device="cuda"))
    return w, x, y, cu, extra


def step(torch, g, w, x, y, cu, extra, H, Hkv, window, loss, plan):
    """Loss value and gradients of x and the weights; bf16 products in torch, the rest the library's."""
    n = x.shape[0]
    qkv = x @ w["qkv"]
    heads = qkv.view(n, H + 2 * Hkv, 128)
    q, k, v = heads[:, :H], heads[:, H:H + Hkv], heads[:, H + Hkv:]
    o = torch.zeros((n, H, 128), dtype=torch.bfloat16, device="cuda")     # rows past the sequences: zeros
    o, lse = g.attention_packed_fwd(q, k, v, plan, o=o)
    h = o.view(n, H * 128) @ w["out"]
    logits = h @ w["head"]
    if loss == "policy":
        out = g.policy_loss(logits, y, extra["old"], extra["adv"], extra["weight"], ref_logp=extra["ref"], kl_coef=0.05,
                            dlogits=logits)
        value, dl = out[0][0], out[2]
    else:
        out = g.preference_loss(logits, y, cu, beta=BETA, dlogits=logits)
        value, dl = out[0], out[4]
        # rows past the sequences are left as they were: logits of 0
    dh = dl @ w["head"].t()
    do = (dh @ w["out"].t()).view(n, H, 128)
    dqkv = torch.zeros_like(qkv)
    dheads = dqkv.view(n, H + 2 * Hkv, 128)
    g.attention_packed_bwd(q, k, v, o, lse, do, plan, dq=dheads[:, :H], dk=dheads[:, H:H + Hkv],
                           dv=dheads[:, H + Hkv:])
    return value, dict(head=h.t() @ dl, out=o.view(n, H * 128).t() @ dh, qkv=x.t() @ dqkv, x=dqkv @ w["qkv"].t())


def exact(torch, w, x, y, cu, extra, H, Hkv, window, loss):
    p = {k: t.double().requires_grad_() for k, t in w.items()}
    xd = x.double().requires_grad_()
    n, total = x.shape[0], int(cu[-1])
    heads = (xd @ p["qkv"]).view(n, H + 2 * Hkv, 128).transpose(0, 1)
    k, v = (t.repeat_interleave(H // Hkv, 0) for t in (heads[H:H + Hkv], heads[H + Hkv:]))
    t = torch.arange(n, device="cuda")
    seq = torch.bucketize(t, cu[1:].long(), right=True)
    seen = (seq[:, None] == seq[None]) & (t[None] <= t[:, None])
    if window >= 0:
        seen &= t[None] >= t[:, None] - window
    P = torch.softmax((heads[:H] @ k.transpose(1, 2) / math.sqrt(128)).masked_fill(~seen, -math.inf), -1)
    o = (P @ v).transpose(0, 1)
    o = torch.where((t < total)[:, None, None], o, 0.0)
    logp = torch.log_softmax(o.reshape(n, -1) @ p["out"] @ p["head"], -1)
    counted = y >= 0
    lp = torch.where(counted, logp.gather(1, y.long().clamp(min=0)[:, None])[:, 0], 0.0)
    if loss == "policy":
        r = torch.exp(lp - extra["old"].double())
        A = extra["adv"].double()
        d = extra["ref"].double() - lp
        each = -torch.minimum(r * A, r.clamp(0.8, 1.2) * A) + 0.05 * (torch.exp(d) - d - 1)
        value = torch.where(counted, each * extra["weight"].double(), 0.0).sum()
    else:
        sums = torch.cat([lp.new_zeros(1), lp.cumsum(0)])
        L = sums[cu[1:].long()] - sums[cu[:-1].long()]
        value = -torch.nn.functional.logsigmoid(BETA * (L[0::2] - L[1::2])).mean()
    value.backward()
    return value.detach(), dict(head=p["head"].grad, out=p["out"].grad, qkv=p["qkv"].grad, x=xd.grad), lp.detach()


@pytest.mark.parametrize("loss", ["policy", "preference"])
@pytest.mark.parametrize("lens,pad,H,Hkv,window", [([37, 150, 1, 90], 20, 2, 1, -1), ([300, 12], 0, 3, 3, 64)])
def test_step(torch, loss, lens, pad, H, Hkv, window):
    import gpt_pretraining_step_b200 as g
    w, x, y, cu, extra = setup(torch, lens, pad, H, Hkv, 1000, len(lens))
    extra["old"], extra["ref"] = torch.zeros_like(extra["adv"]), torch.zeros_like(extra["adv"])

    def near():
        """Other models' log-probabilities near this one's: ratios inside the clip."""
        _, _, lp = exact(torch, w, x, y, cu, extra, H, Hkv, window, loss)
        extra["old"].copy_(lp - 0.1 * torch.tanh(extra["ratio"]))
        extra["ref"].copy_(lp + 0.3 * extra["ratio"])

    def check(value, grads):
        g.op_check()
        want, exact_grads, _ = exact(torch, w, x, y, cu, extra, H, Hkv, window, loss)
        size = float((extra["adv"].abs() * extra["weight"]).sum()) if loss == "policy" else 1.0
        assert abs(float(value) - float(want)) <= BOUND * size
        for name, e in exact_grads.items():
            off = (grads[name].double() - e).norm() / e.norm()
            assert off <= BOUND, (name, float(off))

    near()
    plan = g.attention_plan(cu, x.shape[0], window=window)
    value, grads = step(torch, g, w, x, y, cu, extra, H, Hkv, window, loss, plan)
    check(value, grads)
    # captured, and replayed on another batch of the same size
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(torch, g, w, x, y, cu, extra, H, Hkv, window, loss, plan)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        plan.update(cu)
        value, grads = step(torch, g, w, x, y, cu, extra, H, Hkv, window, loss, plan)
    _, x2, y2, _, _ = setup(torch, lens, pad, H, Hkv, 1000, 77)
    x.copy_(x2)
    y.copy_(y2)
    cu[1] += 3           # other lengths
    near()
    graph.replay()
    check(value, grads)


def brute(torch, q, k, v, lo, rows):
    """o of some rows of one head, in 64 bits."""
    out = []
    for t in rows:
        a = lo(t)
        s = q[t].double() @ k[a:t + 1].double().t() / math.sqrt(128)
        out.append(torch.softmax(s, 0) @ v[a:t + 1].double())
    return torch.stack(out)


@pytest.mark.parametrize("lens,window", [([29] * 5000, -1),                 # more sequences than the plan holds on chip
                                         ([70, 140000, 3], 100),            # more tiles than it has threads
                                         ([1] * 128 * 1030 + [300], -1)])
def test_many_sequences_and_tiles(torch, lens, window):
    import gpt_pretraining_step_b200 as g
    n = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(len(lens))
    q, k, v, do = (torch.randn((n, 1, 128), generator=gen, device="cuda").bfloat16() for _ in range(4))
    starts = np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    plan = g.attention_plan(cu, n, window=window)
    o, lse = g.attention_packed_fwd(q, k, v, plan)
    dq, dk, dv = g.attention_packed_bwd(q, k, v, o, lse, do, plan)
    g.op_check()

    def lo(t):
        a = int(starts[np.searchsorted(starts, t, side="right") - 1])
        return a if window < 0 else max(a, t - window)

    rows = sorted(set(np.random.default_rng(0).integers(0, n, 200).tolist() + [0, 127, 128, n - 1]))
    want = brute(torch, q[:, 0], k[:, 0], v[:, 0], lo, rows)
    got = o[rows, 0].double()
    # P and o rounded to bf16, values of a few
    assert ((got - want).abs() <= 2.0 ** -8 * (want.abs() + 4) + 1e-3).all()
    assert bool(dq.isfinite().all()) and bool(dk.isfinite().all())
    # sum over j of dv_j = sum over t of do_t, as every row of P sums to 1; per
    # element an error of 2^-8 of dv (its rounding, and P's)
    tol = 2 * 2.0 ** -8 * dv.double().abs().sum(0) + 1e-3
    assert ((dv.double().sum(0) - do.double().sum(0)).abs() <= tol).all()


def test_two_captured_graphs_at_once(torch):
    """Two graphs over one plan, replayed side by side on two streams."""
    import gpt_pretraining_step_b200 as g
    lens, n = [400, 90, 22], 512
    cu = torch.tensor([0, 400, 490, 512], dtype=torch.int32, device="cuda")
    plan = g.attention_plan(cu, n)
    sets, alone, graphs, outs = [], [], [], []
    for s in range(2):
        gen = torch.Generator(device="cuda").manual_seed(s)
        t = [torch.randn((n, 4, 128), generator=gen, device="cuda").bfloat16() for _ in range(4)]
        x = torch.randn((n, 3000), generator=gen, device="cuda").bfloat16()
        y = torch.randint(0, 3000, (n,), generator=gen, device="cuda").to(torch.int32)
        sets.append((t, x, y))

    def run(t, x, y):
        o, lse = g.attention_packed_fwd(t[0], t[1], t[2], plan)
        grads = g.attention_packed_bwd(t[0], t[1], t[2], o, lse, t[3], plan)
        ones = torch.ones(n, device="cuda")
        return [o, lse, grads[1], grads[2], *g.policy_loss(x, y, None, ones, ones)]

    for t, x, y in sets:
        alone.append(run(t, x, y))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(t, x, y))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    g.op_check()
    for got, want in zip(outs, alone):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_expired_waits_are_reported_and_calls_recover(torch):
    """A wait limit far below a load's latency: the calls end, GPT_ETIMEOUT is
    reported, and with the usual limit they are right again."""
    import gpt_pretraining_step_b200 as g
    n = 700
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((n, 2, 128), generator=gen, device="cuda").bfloat16() for _ in range(4))
    plan = g.attention_plan(torch.tensor([0, 300, n], dtype=torch.int32, device="cuda"), n)
    o, lse = g.attention_packed_fwd(q, k, v, plan)
    want = [o, lse, *g.attention_packed_bwd(q, k, v, o, lse, do, plan)[1:]]
    g.op_check()
    g.op_set_wait_limit(300)
    try:
        for call in (lambda: g.attention_packed_fwd(q, k, v, plan),
                     lambda: g.attention_packed_bwd(q, k, v, o, lse, do, plan)):
            call()
            with pytest.raises(g.GptError) as e:
                g.op_check()
            assert e.value.code == g.GPT_ETIMEOUT
    finally:
        g.op_set_wait_limit(0)
    o2, lse2 = g.attention_packed_fwd(q, k, v, plan)
    got = [o2, lse2, *g.attention_packed_bwd(q, k, v, o2, lse2, do, plan)[1:]]
    g.op_check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_nothing_to_do(torch):
    """No tokens, no rows: empty results and no error."""
    import gpt_pretraining_step_b200 as g
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    plan = g.attention_plan(cu, 0)
    o, lse = g.attention_packed_fwd(q, k, k, plan)
    dq, dk, dv = g.attention_packed_bwd(q, k, k, o, lse, o, plan)
    g.op_check()
    assert o.shape == q.shape and lse.shape == (4, 0) and dq.shape == q.shape and dk.shape == dv.shape == k.shape
