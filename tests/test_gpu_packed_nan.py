"""A NaN or an infinity in one sequence of a packed batch: the rows that do not
see it (B200 only).

Sequences share tiles of 128 positions, whose products run over all of the tile.
Every row that sees nothing but finite values has to be what it is without the
others: within the bounds of test_gpu_packed_attention (o, lse) and of
test_gpu_packed_gradients (dq, dk, dv), and in tiles that do not visit its tile the
same bit for bit.  Within its own sequence, the rows before it are those of the
sequence cut off there.
"""
import math

import pytest

from test_gpu_packed_attention import reference as forward_reference
from test_gpu_packed_gradients import make, reference

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def run(torch, q, k, v, do, cu, window):
    import gpt_pretraining_step_b200 as g
    plan = g.attention_plan(cu, q.shape[0], window=window)
    o, lse = g.attention_packed_fwd(q, k, v, plan)
    grads = g.attention_packed_bwd(q, k, v, o, lse, do, plan)
    g.op_check()
    return [o, lse.t(), *grads]


def close(torch, got, ref, bounds, what):
    for name, x, r, b in zip("o lse dq dk dv".split(), got, ref, bounds):
        over = (x.double() - r).abs() / (b + 1e-30)
        assert bool(x.isfinite().all()) and float(over.max()) <= 1, (what, name, float(over.max()))


def expected(torch, q, k, v, do, lens, window):
    f = forward_reference(torch, q, k, v, do, lens, window, SCALE)
    grads, errs, _ = reference(torch, q, k, v, do, lens, window, SCALE)
    return [f[0], f[1].t(), *grads], [f[5], f[6].t(), *errs]


CASES = [([40, 50, 30], 1, 10, -1, 2, 1), ([40, 50, 30], 1, 49, -1, 2, 2), ([1, 1, 1, 1], 2, 0, -1, 1, 1),
         ([300, 20, 200, 100], 1, 5, -1, 4, 2), ([300, 20, 200, 100], 0, 290, -1, 2, 2),
         ([500, 130, 7], 1, 100, 60, 3, 1), ([100] * 10, 4, 50, -1, 2, 1)]


@pytest.mark.parametrize("lens,which,at,window,H,Hkv", CASES)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["q", "k", "v", "do", "all"])
def test_rows_that_do_not_see_it(torch, lens, which, at, window, H, Hkv, value, where):
    *t, cu = make(torch, lens, H, Hkv, len(lens) + at)
    t = [x.contiguous() for x in t]
    clean = run(torch, *t, cu, window)
    ref, bounds = expected(torch, *t, lens, window)
    a = sum(lens[:which])
    b, p = a + lens[which], a + at
    for name, x in zip(("q", "k", "v", "do"), t):
        if where in (name, "all"):
            x[p, :, 17 if where != "all" else slice(None)] = value
    got = run(torch, *t, cu, window)
    for rows in (slice(0, a), slice(b, sum(lens))):
        if rows.stop > rows.start:
            close(torch, [x[rows] for x in got], [x[rows] for x in ref], [x[rows] for x in bounds], rows)
    # tiles that do not visit its tile: queries the keys from their first one's on, keys the queries
    # to their last one's (dq's sums have no fixed order)
    n, starts = sum(lens), [sum(lens[:i]) for i in range(len(lens))]
    for at_tile in range(0, n, 128):
        end = min(at_tile + 128, n)
        seq = max(s for s in starts if s <= at_tile)
        first = seq if window < 0 else max(seq, at_tile - window)
        stop = min([s for s in starts if s >= end] + [n])
        final = stop - 1 if window < 0 else min(stop - 1, end - 1 + window)
        rows = slice(at_tile, end)
        if not first // 128 <= p // 128 <= at_tile // 128:
            assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[1][rows], clean[1][rows])
        # of queries all those that see it, whose log-sum-exp and D are others
        if final // 128 < p // 128 or (b - 1) // 128 < at_tile // 128:
            assert torch.equal(got[3][rows], clean[3][rows]) and torch.equal(got[4][rows], clean[4][rows])
    # in its own sequence, the rows before it: outputs and dq do not look ahead
    if at:
        cut = [x[a:p] for x in t]
        ref, bounds = expected(torch, *cut, [at], window)
        close(torch, [got[i][a:p] for i in range(3)], ref[:3], bounds[:3], "before")
    # and its own row is not finite (an infinite score may also be a probability of 0)
    if math.isnan(value):
        assert where == "do" or not got[0][p].isfinite().all()
        assert not got[2][p].isfinite().all()


def test_a_batch_of_nan_alone(torch):
    """Nothing to repair, and quickly seen: every row sees a NaN.  The rows' own
    keys for each would be 17 million steps of a warp."""
    lens = [5000, 3000]
    *t, cu = make(torch, lens, 4, 2, 1)
    for x in t:
        x.fill_(NAN)
    got = run(torch, *t, cu, -1)
    assert all(x.isnan().all() for x in got)
    times = []
    for _ in range(5):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        run(torch, *t, cu, -1)
        end.record()
        end.synchronize()
        times.append(begin.elapsed_time(end))
    assert min(times) < 20, times    # ms; a batch of numbers takes 1
