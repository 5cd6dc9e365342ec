"""Gradients of the packed attention at many sequences and tiles, on two streams,
and with a plan of another batch (B200 only): every row against 64 bits, with the
per-element bounds of test_gpu_packed_gradients, in buffers that held NaN."""
import math

import pytest

from test_gpu_packed_gradients import reference, sequence

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def inputs(torch, n, H, Hkv, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, 2 * H + 2 * Hkv, 128), generator=g, device="cuda").bfloat16()
    return x.split([H, Hkv, Hkv, H], 1)


def offsets(torch, lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def gradients(torch, q, k, v, do, plan):
    """In buffers of NaN: every row has to be written."""
    import gpt_pretraining_step_b200 as g

    def nan(t):
        return torch.full_like(t, math.nan, memory_format=torch.contiguous_format)

    o, lse = g.attention_packed_fwd(q, k, v, plan, o=nan(q),
                                    lse=torch.full((q.shape[1], q.shape[0]), math.nan, device="cuda"))
    got = g.attention_packed_bwd(q, k, v, o, lse, do, plan, dq=nan(q), dk=nan(k), dv=nan(v))
    g.op_check()
    assert o.isfinite().all() and lse.isfinite().all()
    return got


def check(torch, got, want, errs, at=""):
    for name, x, w, e in zip(("dq", "dk", "dv"), got, want, errs):
        over = (x.double() - w).abs() / (e + 1e-30)
        assert float(over.max()) <= 1, (name, at, float(over.max()))    # a NaN fails too


def as_heads(t, count, length):
    """Equal sequences of one head as the heads of one sequence."""
    return t.reshape(count, length, 128).transpose(0, 1)


@pytest.mark.parametrize("count,length,tail", [(5000, 29, 0),              # more sequences than the plan holds on chip
                                               (128 * 1030, 1, 300)])      # and more tiles than it has threads
def test_many_sequences(torch, count, length, tail):
    import gpt_pretraining_step_b200 as g
    n = count * length
    q, k, v, do = inputs(torch, n + tail, 1, 1, count)
    plan = g.attention_plan(offsets(torch, [length] * count + [tail] * (tail > 0)), n + tail)
    got = gradients(torch, q, k, v, do, plan)
    want, errs, _ = sequence(torch, *(as_heads(t[:n], count, length) for t in (q, k, v, do)), -1, SCALE)
    check(torch, [as_heads(t[:n], count, length) for t in got], want, errs)
    if tail:
        want, errs, _ = sequence(torch, *(t[n:] for t in (q, k, v, do)), -1, SCALE)
        check(torch, [t[n:] for t in got], want, errs)


def test_many_tiles_of_one_sequence(torch):
    """More tiles than the plan has threads; a window, so that stretches can be checked by themselves."""
    import gpt_pretraining_step_b200 as g
    lens, window, step = [70, 140000, 3], 100, 2000
    n = sum(lens)
    q, k, v, do = inputs(torch, n, 1, 1, 9)
    got = gradients(torch, q, k, v, do, g.attention_plan(offsets(torch, lens), n, window=window))
    for a, b in ((0, 70), (140070, n)):
        want, errs, _ = sequence(torch, *(t[a:b] for t in (q, k, v, do)), window, SCALE)
        check(torch, [t[a:b] for t in got], want, errs, a)
    for a in range(70, 140070, step):
        # rows from a on see keys from a - window on, and are all that see keys from a on
        first, end = max(70, a - window), min(140070, a + step + window)
        want, errs, _ = sequence(torch, *(t[first:end] for t in (q, k, v, do)), window, SCALE)
        keep = slice(a - first, a - first + step)
        check(torch, [t[a:a + step] for t in got], [w[keep] for w in want], [e[keep] for e in errs], a)


def test_offsets_past_32_bits(torch):
    """More than 2^31 elements in q, o, dq and the fp32 sums: the first and the last sequences."""
    import gpt_pretraining_step_b200 as g
    H, length, count = 16, 500, 2121
    n = length * count
    assert n * H * 128 > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, do = (torch.empty((n, H, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    k, v = (torch.empty((n, 1, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    # head-major q and o, token-major do: both kinds of large strides
    q = q.view(H, n, 128).transpose(0, 1)
    plan = g.attention_plan(torch.arange(0, n + 1, length, dtype=torch.int32, device="cuda"), n)
    o = torch.full((H, n, 128), math.nan, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    o, lse = g.attention_packed_fwd(q, k, v, plan, o=o)
    got = g.attention_packed_bwd(q, k, v, o, lse, do, plan)
    g.op_check()
    for at in (0, 1060, 2119, 2120):
        rows = slice(at * length, (at + 1) * length)
        part = [t[rows] for t in (q, k, v, do)]
        want, errs, _ = sequence(torch, *part, -1, SCALE)
        check(torch, [t[rows] for t in got], want, errs, at)
        again = g.attention_packed_fwd(*(t.contiguous() for t in part[:3]),
                                       g.attention_plan(torch.tensor([0, length], dtype=torch.int32, device="cuda"),
                                                        length))
        # tiles cut the sequence elsewhere there: products add up in another order and P is rounded by another maximum
        assert (again[0].float() - o[rows].float()).abs().max() <= 2.0 ** -6 * 4
        assert (again[1] - lse[:, rows]).abs().max() <= 1e-4
    assert all(bool(t.isfinite().all()) for t in (o, lse, *got))


def test_two_streams(torch):
    """Forward and backward of two batches over one plan at the same time."""
    import gpt_pretraining_step_b200 as g
    lens = [500, 30, 700, 41]
    n = sum(lens)
    sets = [inputs(torch, n, 4, 4, 1), inputs(torch, n, 4, 2, 2)]
    plan = g.attention_plan(offsets(torch, lens), n)
    alone = [gradients(torch, *s, plan) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (q, k, v, do), s in zip(sets, streams):
            o, lse = g.attention_packed_fwd(q, k, v, plan, stream=s)
            got.append(g.attention_packed_bwd(q, k, v, o, lse, do, plan, stream=s))
    torch.cuda.synchronize()
    g.op_check()
    for s, x, w in zip(sets, got, alone):
        assert torch.equal(x[1], w[1]) and torch.equal(x[2], w[2])
        want, errs, _ = reference(torch, *s, lens, -1, SCALE)
        check(torch, x, want, errs)


@pytest.mark.parametrize("planned", [200, 500])
def test_a_plan_of_another_batch_touches_nothing(torch, planned):
    import gpt_pretraining_step_b200 as g
    n = 300
    q, k, v, do = inputs(torch, n, 2, 2, 3)
    plan = g.attention_plan(offsets(torch, [planned // 2, planned - planned // 2]), planned)
    plan.n_tokens = n
    out = [torch.full_like(q, 7.0) for _ in range(4)]
    lse = torch.full((2, n), 7.0, device="cuda")
    for clear in (None, True):
        g.attention_packed_fwd(q, k, v, plan, o=out[0], lse=lse, clear_past=clear)
        with pytest.raises(g.GptError):
            g.op_check()
        g.attention_packed_bwd(q, k, v, q, lse, do, plan, dq=out[1], dk=out[2], dv=out[3], clear_past=clear)
        with pytest.raises(g.GptError):
            g.op_check()
        assert all((t == 7.0).all() for t in (*out, lse))
