"""Performance cases of the fine-tuning operators: attention over packed
sequences, the clipped policy loss and the preference loss.

Each case names an operator, its sizes and its options.  `run` computes one
pass either through the framework's calls (`own` true) or in plain torch
operations in 32 bits; `exact` gives the same results in 64 bits.  Token
counts, head counts and vocabularies are those of this repository's
configurations (32,768 tokens a step at width 1280: 10 heads of 128,
vocabulary 32,768; width 1664: 13 heads; the tiny model's vocabulary of 512)
and odd sizes around them.
"""
import math
import random

import torch

own = False   # set by the caller: True runs the framework's operators

HEAD = 128


def listed():
    return [
        # one short chat message on its own: latency counts
        dict(name="attn fwd one message", op="attention", train=False, tokens=61, shortest=61, longest=61, pad=0,
             heads=10, kv_heads=10, window=-1, layout="heads", lens_seed=1),
        # scoring a batch of chats with a frozen model, grouped kv heads, q|k|v in one projection's rows
        dict(name="attn fwd chats", op="attention", train=False, tokens=16384, shortest=24, longest=1024, pad=0,
             heads=10, kv_heads=2, window=-1, layout="fused", lens_seed=2),
        # one step's tokens of documents up to the context length
        dict(name="attn fwd documents", op="attention", train=False, tokens=32768, shortest=128, longest=2048, pad=0,
             heads=10, kv_heads=10, window=-1, layout="heads", lens_seed=3),
        # fine-tuning on many short examples, padded to a fixed capacity
        dict(name="attn train short", op="attention", train=True, tokens=4001, shortest=1, longest=192, pad=95,
             heads=13, kv_heads=13, window=-1, layout="fused", lens_seed=4),
        # sliding-window layers with grouped kv heads on longer documents
        dict(name="attn train window", op="attention", train=True, tokens=16384, shortest=256, longest=4096, pad=0,
             heads=12, kv_heads=4, window=1024, layout="heads", lens_seed=5),
        # one step's tokens of documents, forward and backward
        dict(name="attn train documents", op="attention", train=True, tokens=32768, shortest=128, longest=2048,
             pad=0, heads=10, kv_heads=10, window=-1, layout="heads", lens_seed=6),
        # a handful of sampled tokens on the tiny vocabulary: latency counts
        dict(name="policy tiny", op="policy", rows=128, vocab=512, ld=512, dtype="bfloat16", masked=0.25, kl=0.04,
             clip_low=0.2, clip_high=0.2),
        # fp32 logits of an odd vocabulary, rows padded to a multiple of 64, no reference model
        dict(name="policy fp32 odd", op="policy", rows=1500, vocab=50257, ld=50304, dtype="float32", masked=0.1,
             kl=0.0, clip_low=0.2, clip_high=0.28),
        # one chunk of lm_head rows of sampled completions, a fifth of the positions (prompts) not counted
        dict(name="policy chunk", op="policy", rows=8192, vocab=32768, ld=32768, dtype="bfloat16", masked=0.2,
             kl=0.02, clip_low=0.2, clip_high=0.2),
        # four short pairs of fp32 logits whose rows are not 16-byte aligned
        dict(name="preference small", op="preference", pairs=4, shortest=5, longest=40, vocab=1001, ld=1001,
             dtype="float32", masked=0.3, beta=0.1, smoothing=0.0, lens_seed=7),
        # a usual step: pairs of chats of some hundred tokens
        dict(name="preference chats", op="preference", pairs=16, shortest=96, longest=512, vocab=32768, ld=32768,
             dtype="bfloat16", masked=0.3, beta=0.1, smoothing=0.0, lens_seed=8),
        # the widest vocabulary, a few long answers, smoothed labels
        dict(name="preference wide", op="preference", pairs=2, shortest=300, longest=900, vocab=131072, ld=131072,
             dtype="bfloat16", masked=0.2, beta=0.3, smoothing=0.1, lens_seed=9),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: Bounds of a drawn case: visible pairs x heads and logits of the largest listed ones.
MOST_SCORES = 1.2e8
MOST_PADDED = 2.4e9
MOST_LOGITS = 2.6e8


def draw(rng):
    op = rng.choice(["attention", "attention", "policy", "preference"])
    if op == "attention":
        while True:
            tokens = _log_uniform(rng, 1, 32768)
            longest = _log_uniform(rng, 1, min(tokens, 8192))
            kv = rng.choice([1, 1, 2, 3, 4, 5, 10, 13])
            heads = kv * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * kv <= 16])
            case = dict(op="attention", train=rng.random() < 0.6, tokens=tokens,
                        shortest=rng.randint(1, max(1, longest // 4)), longest=longest,
                        pad=rng.choice([0, 0, rng.randint(1, 300)]), heads=heads, kv_heads=kv,
                        window=rng.choice([-1, -1, -1, rng.randint(0, 1500)]), layout=rng.choice(["heads", "fused"]),
                        lens_seed=rng.randrange(1 << 30))
            lens = lengths(case)
            if case["train"] and (max(lens) == 1 or case["window"] == 0):
                continue   # every query sees itself alone: dq and dk are zero, with nothing to compare
            if (heads * sum(_visible(n, case["window"]) for n in lens) <= MOST_SCORES
                    and heads * len(lens) * max(lens) ** 2 <= MOST_PADDED):
                return case
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    vocab = _log_uniform(rng, 8, 131072)
    if rng.random() < 0.4:
        vocab = vocab // 8 * 8
    ld = vocab + rng.choice([0, 0, (-vocab) % 64, rng.randint(1, 40)])
    most = MOST_LOGITS / (2 if dtype == "float32" else 1)
    rows = int(max(1, min(8192, most // vocab)))
    if op == "policy":
        return dict(op="policy", rows=_log_uniform(rng, 1, rows), vocab=vocab, ld=ld, dtype=dtype,
                    masked=rng.choice([0.0, rng.uniform(0.05, 0.6)]), kl=rng.choice([0.0, rng.uniform(0.005, 0.2)]),
                    clip_low=rng.uniform(0.1, 0.3), clip_high=rng.uniform(0.1, 0.4))
    pairs = _log_uniform(rng, 1, max(1, min(64, rows // 16)))
    longest = _log_uniform(rng, 2, max(2, min(2048, rows // (2 * pairs))))
    return dict(op="preference", pairs=pairs, shortest=rng.randint(0, max(1, longest // 3)), longest=longest,
                vocab=vocab, ld=ld, dtype=dtype, masked=rng.choice([0.0, rng.uniform(0.05, 0.6)]),
                beta=rng.uniform(0.05, 0.5), smoothing=rng.choice([0.0, rng.uniform(0.01, 0.2)]),
                lens_seed=rng.randrange(1 << 30))


def lengths(case):
    """Sequence lengths of a case: spread over their logarithm; attention fills its tokens."""
    rng = random.Random(case["lens_seed"])
    lo, hi = case["shortest"], case["longest"]
    if case["op"] == "preference":
        lens = [_log_uniform(rng, lo, hi) if lo else rng.randint(0, hi) for _ in range(2 * case["pairs"])]
        return lens if any(lens) else [1] + lens[1:]
    lens, left = [], case["tokens"]
    while left:
        lens.append(min(left, _log_uniform(rng, lo, hi)))
        left -= lens[-1]
    return lens


def _visible(n, window):
    """(query, key) pairs of a causal sequence of n tokens."""
    if window < 0 or window >= n - 1:
        return n * (n + 1) // 2
    w = window + 1
    return w * (w + 1) // 2 + (n - w) * w


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def prepare(case, seed):
    if case["op"] == "attention":
        return _prepare_attention(case, seed)
    return _prepare_loss(case, seed)


def _prepare_attention(case, seed):
    """q and k as the QK norm leaves them (RMS 1 a head), v and the output's
    gradient unit normal; [tokens, heads, 128] views of head-major buffers or
    of the rows of one fused projection."""
    g = _gen(seed)
    lens = lengths(case)
    cu = _cu(lens)
    n, h, hk = cu[-1] + case["pad"], case["heads"], case["kv_heads"]
    x = _randn(g, n, h + 2 * hk, HEAD)
    qk = x[:, :h + hk]
    qk /= qk.square().mean(-1, keepdim=True).sqrt()
    x = x.to(torch.bfloat16)
    q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
    if case["layout"] == "heads":
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    state = dict(case=case, q=q, k=k, v=v, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), total=cu[-1],
                 longest=max(lens))
    if case["train"]:
        state["dout"] = _randn(g, n, h, HEAD).to(torch.bfloat16)
    return state


def _prepare_loss(case, seed):
    """Logits with a spread of 2 and the chosen token well above the rest, as
    trained models give them; log-probabilities of the sampling and the
    reference model near the present ones."""
    g = _gen(seed)
    cu = None
    if case["op"] == "preference":
        cu = _cu(lengths(case))
    m, v = (case["rows"] if cu is None else cu[-1]), case["vocab"]
    x = torch.randn((m, case["ld"]), generator=g, device="cuda", dtype=torch.float32).mul_(2.0)
    targets = torch.randint(0, v, (m,), generator=g, device="cuda")
    at = torch.arange(m, device="cuda")
    x[at, targets] += 2.0 + math.log(v) * _rand(g, m)
    logits = x.to(getattr(torch, case["dtype"]))[:, :v]
    x[:, :v] = logits
    lp = x[at, targets] - torch.logsumexp(x[:, :v], -1)
    del x
    targets = targets.to(torch.int32)
    targets[_rand(g, m) < case["masked"]] = -1
    state = dict(case=case, logits=logits, targets=targets)
    if cu is None:
        # sampled a few updates ago: log ratios of about 0.1, none within 1e-4 of a border
        ratio = 0.12 * _randn(g, m)
        for border in (math.log1p(case["clip_high"]), math.log1p(-case["clip_low"])):
            ratio[(ratio - border).abs() < 1e-4] += 1e-3
        state["old_logp"] = lp - ratio
        state["ref_logp"] = lp + 0.3 * _randn(g, m) if case["kl"] else None
        state["advantage"] = _randn(g, m)
        state["weight"] = (0.5 + _rand(g, m)) / m
        return state
    state["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    counted = torch.where(targets >= 0, lp, 0.0).double()
    sums = torch.cat([counted.new_zeros(1), counted.cumsum(0)])
    seq = sums[state["cu"][1:].long()] - sums[state["cu"][:-1].long()]
    # the reference model's sums: margins of about one
    state["ref_logp"] = (seq + _randn(g, len(seq)) / case["beta"]).float()
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "policy": _own_policy, "preference": _own_preference}[op](state)
    return {"attention": _plain_attention, "policy": _plain_policy, "preference": _plain_preference}[op](state)


# ------------------------------------------------------ the framework's calls

def _own_attention(s):
    import gpt_pretraining_step_b200 as gpt
    n = s["total"]
    plan = gpt.attention_plan(s["cu"], s["q"].shape[0], window=s["case"]["window"])
    o, lse = gpt.attention_packed_fwd(s["q"], s["k"], s["v"], plan)
    out = dict(o=o[:n], lse=lse[:, :n])
    if s["case"]["train"]:
        dq, dk, dv = gpt.attention_packed_bwd(s["q"], s["k"], s["v"], o, lse, s["dout"], plan)
        out.update(dq=dq[:n], dk=dk[:n], dv=dv[:n])
    return out


def _own_policy(s):
    import gpt_pretraining_step_b200 as gpt
    c = s["case"]
    stats, logp, dlogits = gpt.policy_loss(s["logits"], s["targets"], s["old_logp"], s["advantage"], s["weight"],
                                           ref_logp=s["ref_logp"], kl_coef=c["kl"], clip_low=c["clip_low"],
                                           clip_high=c["clip_high"])
    return dict(stats=stats, logp=logp, dlogits=dlogits)


def _own_preference(s):
    import gpt_pretraining_step_b200 as gpt
    c = s["case"]
    loss, margin, seq_logp, logp, dlogits = gpt.preference_loss(
        s["logits"], s["targets"], s["cu"], ref_logp=s["ref_logp"], beta=c["beta"], label_smoothing=c["smoothing"])
    return dict(loss=loss, margin=margin, seq_logp=seq_logp, logp=logp, dlogits=dlogits)


# -------------------------------------------------------------- plain forms

def _plain_attention(s):
    """Sequences padded to the longest: [sequences, heads, longest, 128]."""
    c, cu, n, width = s["case"], s["cu"].long(), s["total"], s["longest"]
    group = c["heads"] // c["kv_heads"]
    at = torch.arange(width, device="cuda")
    valid = at < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + at).clamp(max=n - 1)

    def padded(t):
        return t[rows].float().transpose(1, 2)

    def packed(t, dtype):
        return t.transpose(1, 2)[valid].to(dtype)

    q = padded(s["q"])
    k = padded(s["k"]).repeat_interleave(group, 1)
    v = padded(s["v"]).repeat_interleave(group, 1)
    hidden = at > at[:, None]
    if c["window"] >= 0:
        hidden = hidden | (at < at[:, None] - c["window"])
    scale = 1.0 / math.sqrt(HEAD)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(hidden, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    denom = p.sum(-1, keepdim=True)
    p.div_(denom)
    lse = (top + denom.log())[..., 0]
    o = torch.matmul(p, v)
    out = dict(o=packed(o, torch.bfloat16), lse=lse.transpose(1, 2)[valid].t().contiguous())
    if c["train"]:
        do = torch.where(valid[:, None, :, None], padded(s["dout"]), 0.0)
        dv = torch.matmul(p.transpose(-1, -2), do)
        ds = torch.matmul(do, v.transpose(-1, -2))
        ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dq = torch.matmul(ds, k)
        dk = torch.matmul(ds.transpose(-1, -2), q)
        shape = (len(rows), c["kv_heads"], group, width, HEAD)
        out.update(dq=packed(dq, torch.bfloat16), dk=packed(dk.view(shape).sum(2), torch.bfloat16),
                   dv=packed(dv.view(shape).sum(2), torch.bfloat16))
    return out


def _plain_logp(s):
    """(counted, target or 0, log-probability of the target, softmax)."""
    counted = s["targets"] >= 0
    y = s["targets"].long().clamp(min=0)
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp_()
    denom = p.sum(-1, keepdim=True)
    lp = (x.gather(1, y[:, None]) - top - denom.log())[:, 0]
    p.div_(denom)
    return counted, y, torch.where(counted, lp, 0.0), p


def _plain_dlogits(s, counted, y, p, g):
    """g (1[target] - p), 0 where the row is not counted."""
    g = torch.where(counted, g, 0.0)[:, None]
    d = p.mul_(-g)
    d.scatter_add_(1, y[:, None], g)
    return d.masked_fill_(~counted[:, None], 0.0).to(s["logits"].dtype)


def _plain_policy(s):
    c = s["case"]
    counted, y, lp, p = _plain_logp(s)
    w = torch.where(counted, s["weight"], 0.0)
    a = s["advantage"]
    r = (lp - s["old_logp"]).exp()
    clipped = torch.where(a >= 0, r > 1 + c["clip_high"], r < 1 - c["clip_low"])
    policy = -torch.minimum(r * a, r.clamp(1 - c["clip_low"], 1 + c["clip_high"]) * a)
    g = torch.where(clipped, 0.0, -a * r)
    kl = torch.zeros_like(lp)
    if s["ref_logp"] is not None:
        d = (s["ref_logp"] - lp).double()
        kl = (d.expm1() - d).float()
        g = g - c["kl"] * d.expm1().float()
    terms = torch.stack([policy + c["kl"] * kl, policy, kl, clipped.float()])
    stats = torch.where(counted, terms * w, 0.0).double().sum(1).float()
    return dict(stats=stats, logp=lp, dlogits=_plain_dlogits(s, counted, y, p, g * w))


def _plain_preference(s):
    c, cu = s["case"], s["cu"].long()
    counted, y, lp, p = _plain_logp(s)
    sums = torch.cat([lp.new_zeros(1, dtype=torch.float64), lp.double().cumsum(0)])
    seq = sums[cu[1:]] - sums[cu[:-1]]
    ratio = (seq - s["ref_logp"].double()).view(-1, 2)
    z = c["beta"] * (ratio[:, 0] - ratio[:, 1])
    e = c["smoothing"]
    tail = torch.log1p(torch.exp(-z.abs()))
    loss = ((1 - e) * (z.neg().clamp(min=0) + tail) + e * (z.clamp(min=0) + tail)).mean()
    dz = c["beta"] / len(z) * (e * torch.sigmoid(z) - (1 - e) * torch.sigmoid(-z))
    g = torch.repeat_interleave(torch.stack([dz, -dz], 1).view(-1), cu[1:] - cu[:-1], output_size=len(y)).float()
    return dict(loss=loss.float(), margin=z.float(), seq_logp=seq.float(), logp=lp,
                dlogits=_plain_dlogits(s, counted, y, p, g))


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "policy": _exact_policy, "preference": _exact_preference}[case["op"]](s)


def _exact_attention(s):
    """One sequence after another, in 64 bits."""
    c, n = s["case"], s["total"]
    h, hk = c["heads"], c["kv_heads"]
    f64 = dict(dtype=torch.float64, device="cuda")
    out = dict(o=torch.empty((n, h, HEAD), **f64), lse=torch.empty((h, n), **f64))
    if c["train"]:
        out.update(dq=torch.empty((n, h, HEAD), **f64), dk=torch.empty((n, hk, HEAD), **f64),
                   dv=torch.empty((n, hk, HEAD), **f64))
    edges = s["cu"].tolist()
    head_kv = torch.arange(h, device="cuda") // (h // hk)
    for a, b in zip(edges[:-1], edges[1:]):
        q = s["q"][a:b].double().permute(1, 0, 2)
        k = s["k"][a:b].double().permute(1, 0, 2)[head_kv]
        v = s["v"][a:b].double().permute(1, 0, 2)[head_kv]
        t = torch.arange(b - a, device="cuda")
        gap = t[:, None] - t[None, :]
        seen = gap >= 0
        if c["window"] >= 0:
            seen &= gap <= c["window"]
        score = torch.einsum("hqd,hkd->hqk", q, k) / math.sqrt(HEAD)
        lse = torch.logsumexp(score.masked_fill(~seen, -math.inf), -1)
        p = torch.exp(score - lse[..., None]) * seen
        o = torch.einsum("hqk,hkd->hqd", p, v)
        out["o"][a:b] = o.permute(1, 0, 2)
        out["lse"][:, a:b] = lse
        if not c["train"]:
            continue
        do = s["dout"][a:b].double().permute(1, 0, 2)
        dp = torch.einsum("hqd,hkd->hqk", do, v)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(HEAD)
        out["dq"][a:b] = torch.einsum("hqk,hkd->qhd", ds, k)
        dk, dv = torch.einsum("hqk,hqd->khd", ds, q), torch.einsum("hqk,hqd->khd", p, do)
        out["dk"][a:b] = dk.reshape(b - a, hk, h // hk, HEAD).sum(2)
        out["dv"][a:b] = dv.reshape(b - a, hk, h // hk, HEAD).sum(2)
    return out


def _exact_rows(s):
    x = s["logits"].double()
    y = s["targets"].long()
    seen = y >= 0
    logp = torch.log_softmax(x, -1)
    chosen = torch.zeros_like(x)
    at = seen.nonzero()[:, 0]
    chosen[at, y[at]] = 1.0
    lp = (logp * chosen).sum(-1)
    return seen, lp, chosen.sub_(logp.exp_()).mul_(seen[:, None])


def _exact_policy(s):
    c = s["case"]
    seen, lp, slope = _exact_rows(s)
    w, a = s["weight"].double() * seen, s["advantage"].double()
    lo, hi = 1 - c["clip_low"], 1 + c["clip_high"]
    r = torch.exp(lp - s["old_logp"].double())
    cut = ((a >= 0) & (r > hi)) | ((a < 0) & (r < lo))
    bound = torch.where(a >= 0, torch.full_like(r, hi), torch.full_like(r, lo))
    policy = -a * torch.where(cut, bound, r)
    g = -a * r * ~cut
    kl = torch.zeros_like(lp)
    if s["ref_logp"] is not None:
        d = s["ref_logp"].double() - lp
        kl = torch.exp(d) - d - 1
        g = g + c["kl"] * (1 - torch.exp(d))
    rows = [policy + c["kl"] * kl, policy, kl, cut.double()]
    stats = torch.stack([(w * t)[seen].sum() for t in rows])
    return dict(stats=stats, logp=lp, dlogits=slope * torch.where(seen, w * g, 0.0)[:, None])


def _exact_preference(s):
    c = s["case"]
    seen, lp, slope = _exact_rows(s)
    edges = s["cu"].tolist()
    seq = torch.stack([lp[a:b].sum() for a, b in zip(edges[:-1], edges[1:])])
    over = seq - s["ref_logp"].double()
    z = c["beta"] * (over[0::2] - over[1::2])
    e, pairs = c["smoothing"], c["pairs"]
    logsig = torch.nn.functional.logsigmoid
    loss = -((1 - e) * logsig(z) + e * logsig(-z)).sum() / pairs
    dz = (torch.sigmoid(z) - (1 - e)) * c["beta"] / pairs
    g = torch.zeros_like(lp)
    for i, (a, b) in enumerate(zip(edges[:-1], edges[1:])):
        g[a:b] = dz[i // 2] * (1 if i % 2 == 0 else -1)
    return dict(loss=loss, margin=z, seq_logp=seq, logp=lp, dlogits=slope * g[:, None])


def work(case):
    if case["op"] == "attention":
        lens = lengths(case)
        n, h, hk = sum(lens), case["heads"], case["kv_heads"]
        scores = h * sum(_visible(x, case["window"]) for x in lens)
        qkv = 2 * HEAD * n * (h + 2 * hk)
        moved = qkv + n * h * (2 * HEAD + 4)
        if case["train"]:
            return dict(bytes=moved + 2 * HEAD * n * h + qkv, flops=14 * HEAD * scores)
        return dict(bytes=moved, flops=4 * HEAD * scores)
    size = 4 if case["dtype"] == "float32" else 2
    rows = case["rows"] if case["op"] == "policy" else sum(lengths(case))
    counted = rows * (1 - case["masked"])
    # counted rows are read, every row of the gradient is written; an exponential, a sum and a product per logit
    return dict(bytes=size * case["vocab"] * (counted + rows) + 24 * rows, flops=4 * case["vocab"] * counted)
