"""Attention over packed sequences against the formula in 64 bits (B200 only).

Tolerances are bounds by arithmetic, per element.  With h = 2^-8, the largest
relative error of a rounding to bf16: the kernels round P and dS to bf16 as
matrix operands and the outputs at the end, and read o (rounded) for D.
  o   h (|o| + sum P |v|)
  dv  h (|dv| + sum P |do|)
  dS  2 h |dS| + P sum |do| err(o) (P and dS rounded; D from the rounded o)
  dq  h |dq| + scale sum err(dS) |k|, dk likewise with |q|
each with a share of 2^-12 of the same magnitudes for the fp32 steps.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def make(torch, lens, pad, H, Hkv, layout, seed, garbage=float("nan")):
    """Packed inputs; rows past the last sequence hold `garbage`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = sum(lens)
    n = total + pad
    x = torch.randn((n, 2 * H + 2 * Hkv, 128), generator=g, device="cuda").bfloat16()
    x[total:] = garbage
    q, k, v, do = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:H + 2 * Hkv], x[:, H + 2 * Hkv:]
    if layout == "heads":
        q, k, v, do = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, do))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return q, k, v, do, cu, n


def check(name, got, ref, bound):
    err = (got.double() - ref).abs()
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert torch_isfinite(got), name
    assert worst <= 0, (name, worst, err.max().item(), ref.abs().max().item())


def torch_isfinite(t):
    return bool(t.float().isfinite().all())


def reference(torch, q, k, v, do, lens, window, scale):
    """o, lse, dq, dk, dv and the bound of each, sequence by sequence."""
    H, Hkv = q.shape[1], k.shape[1]
    G = H // Hkv
    out = []
    at = 0
    f32 = 2.0 ** -12
    for n in lens:
        s = slice(at, at + n)
        at += n
        if n == 0:
            continue
        qd, dod = (t[s].double().transpose(0, 1) for t in (q, do))
        kd, vd = (t[s].double().transpose(0, 1).repeat_interleave(G, 0) for t in (k, v))
        t = torch.arange(n, device="cuda")
        hidden = (t[None] > t[:, None]) | (t[None] < t[:, None] - (n if window < 0 else window))
        S = (qd @ kd.transpose(1, 2) * scale).masked_fill(hidden, -math.inf)
        lse = torch.logsumexp(S, -1)
        P = torch.exp(S - lse[..., None])
        o = P @ vd
        e_o = H8 * (o.abs() + P @ vd.abs()) + f32 * (P @ vd.abs())
        e_lse = 2.0 ** -16 * (1 + scale * (qd.abs() @ kd.abs().transpose(1, 2)).amax(-1))
        dP = dod @ vd.transpose(1, 2)
        D = (dod * o).sum(-1, keepdim=True)
        dS = P * (dP - D)
        mag = P * (dod.abs() @ vd.abs().transpose(1, 2) + (dod.abs() * o.abs()).sum(-1, keepdim=True))
        e_dS = 2.02 * H8 * dS.abs() + P * (dod.abs() * e_o).sum(-1, keepdim=True) * (1 + H8) + f32 * mag
        dq, dk, dv = scale * dS @ kd, scale * dS.transpose(1, 2) @ qd, P.transpose(1, 2) @ dod
        e_dq = scale * e_dS @ kd.abs()
        e_dk = scale * e_dS.transpose(1, 2) @ qd.abs()
        e_dv = (H8 + f32) * (P.transpose(1, 2) @ dod.abs())

        def group(x):
            return x.view(Hkv, G, n, 128).sum(1)

        dk, dv, e_dk, e_dv = (group(x) for x in (dk, dv, e_dk, e_dv))
        row = [o, lse, dq, dk, dv, e_o, e_lse, e_dq + H8 * dq.abs(), e_dk + H8 * dk.abs(), e_dv + H8 * dv.abs()]
        out.append([x.transpose(0, 1) if x.dim() == 3 else x for x in row])
    return [torch.cat([r[i] for r in out], 1 if out[0][i].dim() == 2 else 0) for i in range(10)]


def run_and_check(torch, lens, pad, H, Hkv, window, layout, seed=0, scale=0.0):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu, n = make(torch, lens, pad, H, Hkv, layout, seed)
    total = sum(lens)
    mark = 7.0
    plan = g.attention_plan(cu, n, window=window)

    def marked(*shape, dtype=torch.bfloat16):
        return torch.full(shape, mark, dtype=dtype, device="cuda")

    o, lse = g.attention_packed_fwd(q, k, v, plan, scale=scale, o=marked(n, H, 128),
                                    lse=marked(H, n, dtype=torch.float32))
    assert (o[total:] == mark).all() and (lse[:, total:] == mark).all()
    o2 = o.clone()
    o2[total:] = float("nan")
    lse2 = lse.clone()
    lse2[:, total:] = float("nan")
    dq, dk, dv = g.attention_packed_bwd(q, k, v, o2, lse2, do, plan, scale=scale, dq=marked(n, H, 128),
                                        dk=marked(n, Hkv, 128), dv=marked(n, Hkv, 128))
    g.op_check()
    for t in (dq, dk, dv):
        assert (t[total:] == mark).all()
    if not total:
        return
    ref = reference(torch, q, k, v, do, lens, window, scale or 1 / math.sqrt(128))
    got = [o[:total], lse[:, :total], dq[:total], dk[:total], dv[:total]]
    for name, x, r, b in zip("o lse dq dk dv".split(), got, ref[:5], ref[5:]):
        check(name, x, r, b + 1e-30)


LENGTHS = [[1], [2], [127], [128], [129], [255, 1], [1] * 300, [64] * 4, [100, 0, 0, 28, 1, 255, 0], [300, 5, 700],
           [0, 257, 257, 257], [1500], [40, 1200, 3, 3, 900]]


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda x: "-".join(map(str, x[:6])))
@pytest.mark.parametrize("pad,H,Hkv,layout", [(0, 2, 2, "heads"), (1, 3, 1, "fused"), (200, 4, 2, "fused")])
def test_lengths(torch, lens, pad, H, Hkv, layout):
    run_and_check(torch, lens, pad, H, Hkv, -1, layout, seed=sum(lens))


@pytest.mark.parametrize("window", [0, 1, 63, 128, 200, 5000])
@pytest.mark.parametrize("lens", [[1], [130, 300, 7, 1, 513], [1100, 90]], ids=lambda x: "-".join(map(str, x)))
def test_windows(torch, lens, window):
    run_and_check(torch, lens, 33, 2, 1, window, "heads", seed=window + 1)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (13, 13), (10, 5), (16, 1)])
def test_head_splits(torch, H, Hkv):
    run_and_check(torch, [350, 20, 200], 0, H, Hkv, -1, "fused", seed=H)


def test_scale(torch):
    run_and_check(torch, [200, 77], 0, 2, 2, -1, "heads", scale=0.03)


def test_no_sequences(torch):
    run_and_check(torch, [], 150, 2, 2, -1, "heads")
    run_and_check(torch, [0, 0, 0], 10, 2, 2, -1, "heads")


def test_one_sequence_equals_the_unpacked_call(torch):
    """A single full row gives what attention_fwd gives, bit for bit."""
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu, n = make(torch, [700], 0, 4, 2, "heads", 5)
    o, lse = g.attention_packed_fwd(q, k, v, g.attention_plan(cu, n))
    o1, lse1 = g.attention_fwd(*(t.transpose(0, 1)[None].contiguous() for t in (q, k, v)))
    torch.cuda.synchronize()
    assert torch.equal(o, o1[0]) and torch.equal(lse, lse1[0])


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 100], [0, 50, 101], [0, -5, 100], [0, 200, 100]])
def test_bad_offsets_write_nothing(torch, cu):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, _, n = make(torch, [100], 0, 2, 2, "heads", 3)
    plan = g.attention_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n)
    o, lse = torch.full((n, 2, 128), 7.0, device="cuda").bfloat16(), torch.full((2, n), 7.0, device="cuda")
    g.attention_packed_fwd(q, k, v, plan, o=o, lse=lse)
    grads = [torch.full((n, 2, 128), 7.0, device="cuda").bfloat16() for _ in range(3)]
    g.attention_packed_bwd(q, k, v, o, lse, do, plan, dq=grads[0], dk=grads[1], dv=grads[2])
    with pytest.raises(g.GptError) as e:
        g.op_check()
    assert e.value.code == g.GPT_ERANGE
    g.op_check()
    for t in [o, lse] + grads:
        assert (t == 7.0).all()


def test_a_plan_of_another_shape_writes_nothing(torch):
    import gpt_pretraining_step_b200 as g
    q, k, v, _, cu, n = make(torch, [300], 0, 2, 2, "heads", 3)
    plan = g.attention_plan(cu[:1], 200)
    plan.n_tokens = 300
    o = torch.full((n, 2, 128), 7.0, device="cuda").bfloat16()
    g.attention_packed_fwd(q, k, v, plan, o=o)
    with pytest.raises(g.GptError):
        g.op_check()
    assert (o == 7.0).all()


def test_captured_with_new_lengths(torch):
    """A captured plan, forward and backward replay on new offsets and inputs
    in the same buffers."""
    import gpt_pretraining_step_b200 as g
    cases = [[300, 212], [512], [1] * 100 + [17, 200]]
    n = 512
    q, k, v, do, cu, _ = make(torch, [n], 0, 2, 2, "fused", 0)
    offsets = torch.zeros(200, dtype=torch.int32, device="cuda")
    offsets[1:] = n
    plan = g.attention_plan(offsets, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = g.attention_packed_fwd(q, k, v, plan)
        g.attention_packed_bwd(q, k, v, o, lse, do, plan)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.update(offsets)
        o, lse = g.attention_packed_fwd(q, k, v, plan)
        dq, dk, dv = g.attention_packed_bwd(q, k, v, o, lse, do, plan)
    for i, lens in enumerate(cases):
        total = sum(lens)
        q1, k1, v1, do1, cu1, _ = make(torch, lens, n - total, 2, 2, "fused", 10 + i)
        for a, b in ((q, q1), (k, k1), (v, v1), (do, do1)):
            a.copy_(b)
        offsets.fill_(total)
        offsets[:len(cu1)] = cu1
        graph.replay()
        g.op_check()
        ref = reference(torch, q1, k1, v1, do1, lens, -1, 1 / math.sqrt(128))
        for name, x, r, b in zip("o lse dq dk dv".split(),
                                 [o[:total], lse[:, :total], dq[:total], dk[:total], dv[:total]], ref[:5], ref[5:]):
            check(name, x, r, b + 1e-30)


def test_two_streams_share_a_plan(torch):
    import gpt_pretraining_step_b200 as g
    lens = [500, 30, 700, 41]
    a = make(torch, lens, 0, 4, 4, "heads", 1)
    b = make(torch, lens, 0, 4, 2, "fused", 2)
    plan = g.attention_plan(a[4], a[5])
    alone = [g.attention_packed_fwd(x[0], x[1], x[2], plan) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [g.attention_packed_fwd(x[0], x[1], x[2], plan, stream=s) for x, s in zip((a, b), streams)]
        grads = [g.attention_packed_bwd(x[0], x[1], x[2], o, lse, x[3], plan, stream=s)
                 for x, (o, lse), s in zip((a, b), got, streams)]
    torch.cuda.synchronize()
    g.op_check()
    for (o, lse), (o1, lse1) in zip(got, alone):
        assert torch.equal(o, o1) and torch.equal(lse, lse1)
    assert all(torch_isfinite(t) for ts in grads for t in ts)


def test_strides_and_views(torch):
    """Inputs, outputs and gradients in slices of wider buffers, which stay as
    they were around the slices."""
    import gpt_pretraining_step_b200 as g
    lens, H, n = [150, 90], 2, 240
    q, k, v, do, cu, _ = make(torch, lens, 0, H, H, "heads", 9)
    o, lse = g.attention_packed_fwd(q, k, v, g.attention_plan(cu, n))
    wide = torch.full((n + 2, H + 3, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    ow = wide[1:-1, 1:1 + H, 8:]
    g.attention_packed_fwd(q, k, v, g.attention_plan(cu, n), o=ow, lse=lse)
    assert torch.equal(ow, o)
    wide[1:-1, 1:1 + H, 8:] = 7.0
    assert (wide == 7.0).all()
    dqkv = torch.full((n, 3 * H + 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = g.attention_plan(cu, n)
    g.attention_packed_bwd(q, k, v, o, lse, do, plan, dq=dqkv[:, :H], dk=dqkv[:, H:2 * H], dv=dqkv[:, 2 * H:3 * H])
    g.op_check()
    ref = reference(torch, q, k, v, do, lens, -1, 1 / math.sqrt(128))
    for i in range(3):
        check("dqkv"[i + 1], dqkv[:, i * H:(i + 1) * H], ref[2 + i], ref[7 + i] + 1e-30)
    assert (dqkv[:, 3 * H:] == 7.0).all()
    one = torch.randn((1, 1, 128), device="cuda").bfloat16()   # extent-1 dimensions: any stride
    o1, _ = g.attention_packed_fwd(one.as_strided((1, 1, 128), (3, 5, 1)), one, one,
                                   g.attention_plan(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1))
    assert torch.equal(o1, one)


def test_refusals(torch):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu, n = make(torch, [64], 0, 4, 2, "heads", 3)
    plan = g.attention_plan(cu, n)
    o, lse = g.attention_packed_fwd(q, k, v, plan)
    bad = [lambda: g.attention_packed_fwd(q.float(), k, v, plan), lambda: g.attention_packed_fwd(q[:-1], k, v, plan),
           lambda: g.attention_packed_fwd(q[:, :3], k, v, plan), lambda: g.attention_packed_fwd(q, k, v[:, :1], plan),
           lambda: g.attention_packed_fwd(q.cpu(), k, v, plan), lambda: g.attention_packed_fwd(q, k.cpu(), v, plan),
           lambda: g.attention_packed_fwd(q, k, v, plan, scale=-1.0),
           lambda: g.attention_packed_fwd(q, k, v, plan, scale=math.inf),
           lambda: g.attention_packed_fwd(q, k, v, plan, o=o[:, :1].expand(-1, 4, -1)),
           lambda: g.attention_packed_fwd(q, k, v, plan, lse=lse.half()),
           lambda: g.attention_packed_bwd(q, k, v, o, lse, do[:, :2], plan),
           lambda: g.attention_packed_bwd(q, k, v, o, lse[:, :-1], do, plan),
           lambda: g.attention_plan(cu.long(), n), lambda: g.attention_plan(cu.cpu(), n),
           lambda: g.attention_plan(cu, -1)]
    for i, call in enumerate(bad):
        with pytest.raises(g.GptError) as e:
            call()
        assert e.value.code == g.GPT_EINVAL, i
    g.op_check()


def test_plan_of_another_device(torch):
    """Memory of one device is not read by another's kernels."""
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu, n = make(torch, [64], 0, 4, 2, "heads", 3)
    plan = g.attention_plan(cu, n)
    o, lse = g.attention_packed_fwd(q, k, v, plan)
    plan.device = 1   # as if it had been made there
    for call in (lambda: g.attention_packed_fwd(q, k, v, plan), lambda: plan.update(cu),
                 lambda: g.attention_packed_bwd(q, k, v, o, lse, do, plan)):
        with pytest.raises(g.GptError, match="cuda:1"):
            call()
    g.op_check()


def test_windows_past_32_bits_are_no_window(torch):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu, n = make(torch, [200, 57], 0, 2, 2, "heads", 4)
    want = g.attention_packed_fwd(q, k, v, g.attention_plan(cu, n))
    for window in (2 ** 40, 2 ** 32, 2 ** 31 - 1, -2 ** 40):
        got = g.attention_packed_fwd(q, k, v, g.attention_plan(cu, n, window))
        assert all(torch.equal(a, b) for a, b in zip(want, got)), window
    g.op_check()
