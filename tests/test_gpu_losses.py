"""Policy and preference losses against their formulas in 64 bits (B200 only).

Tolerances: the exponentials, their sum and the log are fp32 (relative steps
of 2^-24 to 2^-22, an argument x - m of up to about 100 rounded once more), so
a log-probability is off by at most 4e-6 + 2^-22 |lp| and a probability by
2e-5 of itself; a gradient value then by 3e-5 of G (p + 1[target]), G the sum
of the magnitudes in its row factor, plus for bf16 the rounding 2^-8.
"""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def make_rows(torch, M, V, dtype, ld, masked, seed, base=0):
    """Logits as a view at `base` elements into a buffer of rows of ld."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, V), generator=g, device="cuda") * 2
    y = torch.randint(0, V, (M,), generator=g, device="cuda")
    x[torch.arange(M, device="cuda"), y] += 3.0
    buf = torch.full((M * ld + base,), float("nan"), dtype=dtype, device="cuda")
    logits = buf[base:].as_strided((M, V), (ld, 1))
    logits.copy_(x)
    y = y.to(torch.int32)
    y[torch.rand(M, generator=g, device="cuda") < masked] = -1
    return logits, y, g


def exact_rows(torch, logits, y):
    x = logits.double()
    lp_all = torch.log_softmax(x, -1)
    seen = y >= 0
    t = y.long().clamp(min=0)[:, None]
    lp = torch.where(seen, lp_all.gather(1, t)[:, 0], 0.0)
    hot = torch.zeros_like(x).scatter_(1, t, 1.0)
    return seen, lp, lp_all.exp(), hot


def check_lp(torch, got, lp):
    assert ((got.double() - lp).abs() <= 4e-6 + 2.0 ** -22 * lp.abs()).all()


def check_grad(torch, got, seen, g, G, p, hot):
    ref = torch.where(seen[:, None], g[:, None] * (hot - p), 0.0)
    bound = torch.where(seen[:, None], 3e-5 * G[:, None] * (p + hot), 0.0)
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ref.abs() * (1 + 1e-4)
    # results under the smallest normal number are flushed or rounded to steps of it
    err = (got.double() - ref).abs()
    assert (err <= bound + 1.2e-38).all(), (err - bound).max().item()


ROWS = [(1, 1, "float32", 1, 0), (5, 7, "bfloat16", 7, 0), (64, 512, "bfloat16", 512, 0), (33, 1001, "float32", 1001, 1),
        (40, 1001, "bfloat16", 1003, 3), (300, 1000, "bfloat16", 1024, 0), (9, 50257, "float32", 50304, 0),
        (12, 32768, "bfloat16", 32768, 0), (5, 131072, "bfloat16", 131072, 0), (3, 131071, "float32", 131071, 2),
        (2, 300001, "bfloat16", 300001, 1)]


@pytest.mark.parametrize("M,V,dtype,ld,base", ROWS)
@pytest.mark.parametrize("kl,old", [(0.0, True), (0.1, True), (0.05, False)])
def test_policy_loss(torch, M, V, dtype, ld, base, kl, old):
    import gpt_pretraining_step_b200 as gpt
    logits, y, gen = make_rows(torch, M, V, getattr(torch, dtype), ld, 0.3, M + V, base)
    seen, lp, p, hot = exact_rows(torch, logits, y)
    ratio = torch.randn(M, generator=gen, device="cuda") * 0.2
    lo, hi = 0.25, 0.5                      # exact in fp32
    for b in (math.log(1 + hi), math.log(1 - lo)):
        ratio[(ratio - b).abs() < 1e-3] += 3e-3
    old_lp = (lp.float() - ratio) if old else None
    ref_lp = lp.float() + 0.5 * torch.randn(M, generator=gen, device="cuda") if kl else None
    if kl:
        ref_lp[0] = lp[0].float()            # a difference near zero
    adv = torch.randn(M, generator=gen, device="cuda")
    adv[M // 2] = 0.0
    w = torch.rand(M, generator=gen, device="cuda") / M
    w[M // 3] = 0.0
    seen = seen & (w != 0)
    stats, logp, d = gpt.policy_loss(logits, y, old_lp, adv, w, ref_logp=ref_lp, kl_coef=kl, clip_low=lo, clip_high=hi)
    gpt.op_check()
    lp = torch.where(seen, lp, 0.0)
    check_lp(torch, logp, lp)
    A, W = adv.double(), torch.where(seen, w.double(), 0.0)
    r = torch.exp(lp - old_lp.double()) if old else torch.ones_like(lp)
    cut = torch.where(A >= 0, r > 1 + hi, r < 1 - lo)
    surrogate = -torch.minimum(r * A, r.clamp(1 - lo, 1 + hi) * A)
    dd = ref_lp.double() - lp if kl else torch.zeros_like(lp)
    k = torch.expm1(dd) - dd
    g = W * (torch.where(cut, 0.0, -A * r) - kl * torch.expm1(dd))
    G = W * (A.abs() * r + kl * (torch.exp(dd) + 1))
    want = torch.stack([W * (surrogate + kl * k), W * surrogate, W * k, W * cut])
    size = torch.stack([W * (A.abs() * r + kl * (torch.exp(dd) + 1)), W * A.abs() * r, W * (torch.exp(dd) + 1), W])
    size = torch.where(seen, size, 0.0)
    assert ((stats.double() - torch.where(seen, want, 0.0).sum(1)).abs() <= 2e-5 * size.sum(1)).all()
    check_grad(torch, d, seen, g, G, p, hot)
    # the same in place, without a gradient, and again: bit for bit
    s2, l2, none = gpt.policy_loss(logits, y, old_lp, adv, w, ref_logp=ref_lp, kl_coef=kl, clip_low=lo, clip_high=hi,
                                   grad=False)
    assert none is None and torch.equal(s2, stats) and torch.equal(l2, logp)
    keep = d.clone()
    _, _, d3 = gpt.policy_loss(logits, y, old_lp, adv, w, ref_logp=ref_lp, kl_coef=kl, clip_low=lo, clip_high=hi,
                               dlogits=logits)
    assert d3 is logits and torch.equal(d3, keep)


@pytest.mark.parametrize("M,V,dtype,ld,base", [r for r in ROWS if r[0] > 2])
@pytest.mark.parametrize("smoothing,ref", [(0.0, True), (0.2, False)])
def test_preference_loss(torch, M, V, dtype, ld, base, smoothing, ref):
    import gpt_pretraining_step_b200 as gpt
    logits, y, gen = make_rows(torch, M, V, getattr(torch, dtype), ld, 0.3, M + V, base)
    lens = [M // 3, M // 4, 0, M // 5 + 1]
    total = sum(lens)
    cu = torch.tensor([0, lens[0], lens[0] + lens[1], lens[0] + lens[1], total], dtype=torch.int32, device="cuda")
    logits[total:] = float("nan")
    beta = 0.25
    seen, lp, p, hot = exact_rows(torch, logits[:total], y[:total])
    edges = cu.tolist()
    L = torch.stack([lp[a:b].sum() for a, b in zip(edges[:-1], edges[1:])])
    R = (L + 3 * torch.randn(4, generator=gen, device="cuda")).float() if ref else None
    d = torch.full_like(logits, 7.0)
    loss, margin, seq, logp, d = gpt.preference_loss(logits, y, cu, ref_logp=R, beta=beta, label_smoothing=smoothing,
                                                     dlogits=d)
    gpt.op_check()
    check_lp(torch, logp[:total], lp)
    over = L - (R.double() if ref else 0.0)
    z = beta * (over[0::2] - over[1::2])
    ls = torch.nn.functional.logsigmoid
    want = (-(1 - smoothing) * ls(z) - smoothing * ls(-z)).mean()
    dz = beta / 2 * (smoothing * torch.sigmoid(z) - (1 - smoothing) * torch.sigmoid(-z))
    e_L = 4e-6 * M + 2.0 ** -22 * L.abs().sum()
    assert ((seq.double() - L).abs() <= e_L).all()
    assert ((margin.double() - z).abs() <= 2 * beta * e_L + 2.0 ** -23 * z.abs()).all()
    assert abs(loss.double() - want) <= 2 * beta * e_L + 2.0 ** -23 * want
    per = torch.stack([dz, -dz], 1).view(-1)
    g = torch.cat([per[i].expand(n) for i, n in enumerate(lens)])
    slack = beta * beta * e_L * torch.ones_like(g)      # a sigmoid changes by at most its argument's error
    check_grad(torch, d[:total], seen, g, g.abs() + slack / 3e-5, p, hot)
    assert (d[total:] == 7.0).all()
    again = gpt.preference_loss(logits, y, cu, ref_logp=R, beta=beta, label_smoothing=smoothing, grad=False)
    assert again[4] is None and torch.equal(again[0], loss) and torch.equal(again[2], seq)
    keep = d[:total].clone()
    inplace = gpt.preference_loss(logits, y, cu, ref_logp=R, beta=beta, label_smoothing=smoothing, dlogits=logits)
    assert torch.equal(inplace[4][:total], keep) and inplace[4][total:].isnan().all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_masked_logits_and_rows(torch, dtype):
    """-inf and the type's lowest value as masks, a huge row, rows of NaN that
    are not counted, and a row whose every value is the lowest."""
    import gpt_pretraining_step_b200 as gpt
    M, V = 8, 5000
    dt = getattr(torch, dtype)
    logits, y, _ = make_rows(torch, M, V, dt, V, 0.0, 5)
    low = torch.finfo(dt).min
    y[:] = 17
    logits[0, 100:] = -math.inf
    logits[1, 100:] = low
    logits[2] = float("nan")
    y[2] = -1
    logits[3] = low
    logits[4] = logits[4] * 0 + 3e38
    logits[5, :4096] = -math.inf
    y[5] = 4999
    logits[6] = math.inf
    w = torch.ones(M, device="cuda")
    w[6] = 0.0
    adv = torch.ones(M, device="cuda")
    stats, logp, d = gpt.policy_loss(logits, y, None, adv, w)
    gpt.op_check()
    seen, lp, p, hot = exact_rows(torch, logits, y)
    seen = seen & (w != 0)
    ok = torch.where(seen, lp, 0.0)
    check_lp(torch, logp, ok)
    check_grad(torch, d, seen, -torch.ones_like(lp), torch.ones_like(lp), torch.where(seen[:, None], p, 0.0), hot)
    assert (d[2] == 0).all() and (d[6] == 0).all() and (d[0, 100:] == 0).all()
    assert stats[0] == -float(seen.sum())


def test_ids_out_of_range_are_not_counted(torch):
    import gpt_pretraining_step_b200 as gpt
    logits, y, _ = make_rows(torch, 6, 50, torch.float32, 50, 0.0, 1)
    y[1], y[4] = 50, -2
    ones = torch.ones(6, device="cuda")
    _, logp, d = gpt.policy_loss(logits, y, None, ones, ones)
    with pytest.raises(gpt.GptError) as e:
        gpt.op_check()
    assert e.value.code == gpt.GPT_ERANGE
    assert (d[1] == 0).all() and (d[4] == 0).all() and logp[1] == 0 and logp[4] == 0 and (d[0] != 0).all()


@pytest.mark.parametrize("cu", [[0, 4, 2], [1, 4, 6], [0, 3, 7], [0, 9, 6]])
def test_bad_offsets_write_nothing(torch, cu):
    import gpt_pretraining_step_b200 as gpt
    logits, y, _ = make_rows(torch, 6, 50, torch.float32, 50, 0.0, 1)
    d = torch.full_like(logits, 7.0)
    gpt.preference_loss(logits, y, torch.tensor(cu, dtype=torch.int32, device="cuda"), dlogits=d)
    with pytest.raises(gpt.GptError) as e:
        gpt.op_check()
    assert e.value.code == gpt.GPT_ERANGE
    assert (d == 7.0).all()


def test_empty(torch):
    import gpt_pretraining_step_b200 as gpt
    logits = torch.empty((0, 100), device="cuda")
    none = torch.empty(0, device="cuda")
    stats, logp, d = gpt.policy_loss(logits, torch.empty(0, dtype=torch.int32, device="cuda"), none, none, none)
    loss, margin, seq, logp, d = gpt.preference_loss(logits, torch.empty(0, dtype=torch.int32, device="cuda"),
                                                     torch.zeros(5, dtype=torch.int32, device="cuda"))
    gpt.op_check()
    assert (stats == 0).all() and (margin == 0).all() and abs(float(loss) - math.log(2)) < 1e-6


def test_gradient_by_differences(torch):
    """The whole gradient of both losses against central differences of their
    own loss values, along random directions, in fp32."""
    import gpt_pretraining_step_b200 as gpt
    M, V, step = 24, 64, 2.0 ** -6
    logits, y, gen = make_rows(torch, M, V, torch.float32, V, 0.2, 3)
    _, lp, _, _ = exact_rows(torch, logits, y)
    lp = lp.float()
    adv = torch.randn(M, generator=gen, device="cuda")
    w = torch.rand(M, generator=gen, device="cuda")
    cu = torch.tensor([0, 9, 13, 20, 24], dtype=torch.int32, device="cuda")
    # ratios well inside the clip, so that no border is crossed
    calls = [lambda x: gpt.policy_loss(x, y, lp - 0.1, adv, w, ref_logp=lp + 0.3, kl_coef=0.5, clip_low=0.9,
                                       clip_high=9.0)[::2],
             lambda x: gpt.preference_loss(x, y, cu, beta=0.2, label_smoothing=0.1)[::4]]
    for call in calls:
        _, d = call(logits)
        for _ in range(4):
            u = torch.randn((M, V), generator=gen, device="cuda")
            u /= u.norm()
            ends = [call(logits + s * u)[0].reshape(-1)[0].double() for s in (step, -step)]
            slope = (ends[0] - ends[1]) / (2 * step)
            # the loss is rounded to fp32 (2^-23 of up to ~10) and the third
            # derivative along a unit direction is below ~10
            assert abs(slope - (d.double() * u).sum()) <= 10 * 2.0 ** -23 * 4 / step + 10 * step ** 2 / 6


def test_captured_and_two_streams(torch):
    import gpt_pretraining_step_b200 as gpt
    sets = [make_rows(torch, 40, 3000, torch.bfloat16, 3000, 0.2, s) for s in range(3)]
    cu = torch.tensor([0, 10, 25, 32, 40], dtype=torch.int32, device="cuda")
    adv, w = torch.randn(40, device="cuda"), torch.rand(40, device="cuda")

    def both(x, y, stream=None):
        return list(gpt.policy_loss(x, y, None, adv, w, stream=stream)) + list(
            gpt.preference_loss(x, y, cu, stream=stream))

    want = [both(x, y) for x, y, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [both(x, y, s) for (x, y, _), s in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    x, y = sets[0][0].clone(), sets[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x, y)
    for (x1, y1, _), b in zip(sets, want):
        x.copy_(x1)
        y.copy_(y1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(out, b))
    gpt.op_check()


def test_refusals(torch):
    import gpt_pretraining_step_b200 as gpt
    x, y, _ = make_rows(torch, 8, 40, torch.float32, 40, 0.0, 1)
    a = torch.ones(8, device="cuda")
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    bad = [lambda: gpt.policy_loss(x.half(), y, a, a, a), lambda: gpt.policy_loss(x, y.long(), a, a, a),
           lambda: gpt.policy_loss(x, y[:-1], a, a, a), lambda: gpt.policy_loss(x, y, a.double(), a, a),
           lambda: gpt.policy_loss(x, y, a, a[:-1], a), lambda: gpt.policy_loss(x.cpu(), y, a, a, a),
           lambda: gpt.policy_loss(x.t(), y, a, a, a), lambda: gpt.policy_loss(x, y, a, a, a, kl_coef=0.1),
           lambda: gpt.policy_loss(x, y, a, a, a, clip_low=1.5), lambda: gpt.policy_loss(x, y, a, a, a, clip_high=-0.1),
           lambda: gpt.policy_loss(x, y, a, a, a, clip_high=math.nan),
           lambda: gpt.policy_loss(x, y, a, a, a, dlogits=x.bfloat16()),
           lambda: gpt.policy_loss(x, y, a, a, a, dlogits=x[:4]),
           lambda: gpt.preference_loss(x, y, cu[:2]), lambda: gpt.preference_loss(x, y, cu.long()),
           lambda: gpt.preference_loss(x, y, cu, ref_logp=a), lambda: gpt.preference_loss(x, y, cu, beta=math.inf),
           lambda: gpt.preference_loss(x, y, cu, label_smoothing=1.1),
           lambda: gpt.policy_loss(x[:1].expand(8, -1), y, a, a, a)]
    for i, call in enumerate(bad):
        with pytest.raises(gpt.GptError) as e:
            call()
        assert e.value.code == gpt.GPT_EINVAL, i
    gpt.op_check()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_errors_of_log_probabilities_do_not_add_up(torch, dtype):
    """Their mean over many rows, which a sequence's sum multiplies by its
    length: the exponentials' mean error is made up for to 2.8e-8 at worst
    (where the argument is above -1), and 8192 errors of 2.5e-7 root mean square
    average to within 3 * 2.8e-9."""
    import gpt_pretraining_step_b200 as gpt
    off = []
    for seed in range(4):
        logits, y, _ = make_rows(torch, 2048, 20000, getattr(torch, dtype), 20000, 0.0, seed)
        cu = torch.tensor([0, 2048, 2048], dtype=torch.int32, device="cuda")
        _, _, seq, logp, _ = gpt.preference_loss(logits, y, cu, grad=False)
        _, lp, _, _ = exact_rows(torch, logits, y)
        off.append(logp.double() - lp)
        # the sum is rounded once more
        most = 2048 * (2.8e-8 + 3 * 2.5e-7 / 2048 ** 0.5) + 2.0 ** -24 * lp.sum().abs()
        assert abs(seq[0].double() - lp.sum()) <= most
    assert abs(torch.cat(off).mean()) <= 2.8e-8 + 3 * 2.8e-9


def test_infinite_terms_of_weight_zero(torch):
    """A counted target masked to -inf: lp = -inf, so the KL estimate is infinite
    and an answer's sum, too; where their weights are 0 they are no part of the
    loss, and the gradients stay finite."""
    import gpt_pretraining_step_b200 as gpt
    M, V = 4, 300
    logits, y, _ = make_rows(torch, M, V, torch.float32, V, 0.0, 3)
    logits[3, y[3].long()] = -math.inf
    one, old = torch.ones(M, device="cuda"), torch.zeros(M, device="cuda")
    ref = torch.full((M,), -2.0, device="cuda")
    stats, logp, d = gpt.policy_loss(logits, y, old, one, one, ref_logp=ref, kl_coef=0.0)
    want, _, want_d = gpt.policy_loss(logits, y, old, one, one)
    assert logp[3] == -math.inf and stats[2] == math.inf
    assert torch.equal(stats[:2], want[:2]) and stats[0].isfinite()
    assert torch.equal(d, want_d) and (d[3] == 0).all() and d.isfinite().all()
    # the rejected answer is impossible: the margin is infinite and nothing is left to learn
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    loss, margin, seq, _, d = gpt.preference_loss(logits, y, cu)
    assert loss == 0 and margin[0] == math.inf and seq[1] == -math.inf and (d == 0).all()
    # the chosen one is
    cu = torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda")
    loss, margin, _, _, d = gpt.preference_loss(logits[2:], y[2:], cu, beta=0.5)
    assert loss == math.inf and margin[0] == -math.inf and d.isfinite().all()
    gpt.op_check()


def test_new_gradient_leaves_out_the_gaps(torch):
    """Of logits that are every tenth row of a buffer: rows as aligned, memory
    of the rows alone."""
    import gpt_pretraining_step_b200 as gpt
    for dt, n in ((torch.bfloat16, 8), (torch.float32, 4)):
        for V, ld in ((1000, 10000), (1001, 10008), (1001, 10010)):
            logits, y, _ = make_rows(torch, 6, V, dt, ld, 0.0, 3)
            one = torch.ones(6, device="cuda")
            _, _, d = gpt.policy_loss(logits, y, None, one, one)
            _, _, flat = gpt.policy_loss(logits.contiguous(), y, None, one, one)
            assert V <= d.stride(0) < V + n and (d.stride(0) - ld) % n == 0
            assert d.untyped_storage().nbytes() <= 6 * d.stride(0) * d.element_size()
            assert torch.allclose(d, flat, rtol=2.0 ** -7, atol=1e-6)
    gpt.op_check()
