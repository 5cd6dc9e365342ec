"""How accurate the gradients of the packed attention are (B200 only).

Two kinds of tolerance, h = 2^-8 being the largest relative error of a
rounding to bf16.

Per element, from the formulas: of the operands only dS (for dq and dk) and P
(for dv) are rounded to bf16, and the results once more.  Everything else is
fp32: a sum of n products is off by at most f(n) = max(n, 128) 2^-23 of the sum
of their magnitudes (every addition truncated), which for the scores S makes
  P   e_P = 2 scale f |q|.|k| + 2^-18 of itself (its own score's error and the
      log-sum-exp's, the exponentials and the scaling)
  dP  f |do|.|v|
  D   sum P (f |do|.|v| + 2 e_P |dP - D|), as D is divided by the sum of P
  dS  (h + e_P) |dS| + P (err(dP) + err(D))
  dq  h |dq| + scale (sum err(dS) |k| + f sum |dS| |k|), dk likewise with |q|
  dv  h |dv| + sum (h + e_P + f) P |do|

In the 2-norm: a rounding to bf16 is uniform within half a step, 2^-8 / sqrt(3)
of the value at the start of a binade, and 0.7355 of that averaged over a
binade's logarithm: 0.00166 root mean square.  Independent roundings of dS (or P)
and of the result add up to 0.00166 sqrt(1 + C^2), C^2 = sum dS^2 |k|^2 scale^2 /
|dq|^2; a quarter more is allowed for the number of values.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8
RMS = 0.00166


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def fp32_sum(n):
    return max(n, 128) * 2.0 ** -23


def make(torch, lens, H, Hkv, seed):
    """q and k of RMS 1 a head, as the QK norm leaves them; v and do unit normal."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lens)
    x = torch.randn((n, 2 * H + 2 * Hkv, 128), generator=g, device="cuda")
    x[:, :H + Hkv] /= x[:, :H + Hkv].square().mean(-1, keepdim=True).sqrt()
    x = x.bfloat16()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return (*x.split([H, Hkv, Hkv, H], 1), cu)


def sequence(torch, q, k, v, do, window, scale):
    """Gradients of one sequence in 64 bits, the bound of each element, and
    the squares of what the roundings of dS make of dq and dk."""
    n, H, Hkv = q.shape[0], q.shape[1], k.shape[1]
    G = H // Hkv
    qd, dod = (t.double().transpose(0, 1) for t in (q, do))
    kd, vd = (t.double().transpose(0, 1).repeat_interleave(G, 0) for t in (k, v))
    t = torch.arange(n, device="cuda")
    hidden = (t[None] > t[:, None]) | (t[None] < t[:, None] - (n if window < 0 else window))
    S = (qd @ kd.transpose(1, 2) * scale).masked_fill(hidden, -math.inf)
    P = torch.softmax(S, -1)
    dP = dod @ vd.transpose(1, 2)
    D = (P * dP).sum(-1, keepdim=True)
    dS = P * (dP - D)
    f = fp32_sum(n)
    e_P = 2 * scale * f * (qd.abs() @ kd.abs().transpose(1, 2)).amax(-1, keepdim=True) + 2.0 ** -18
    e_dP = f * (dod.abs() @ vd.abs().transpose(1, 2))
    e_D = (P * (e_dP + 2 * e_P * (dP - D).abs())).sum(-1, keepdim=True)
    e_dS = (H8 + e_P) * dS.abs() + P * (e_dP + e_D)
    to_k, size = dS.transpose(1, 2), dS.abs()

    def group(x):
        return x.view(Hkv, G, n, 128).sum(1)

    grads = [scale * dS @ kd, group(scale * to_k @ qd), group(P.transpose(1, 2) @ dod)]
    f *= G
    errs = [scale * (e_dS + f * size) @ kd.abs(), group(scale * (e_dS + f * size).transpose(1, 2) @ qd.abs()),
            group((P * (H8 + e_P + f)).transpose(1, 2) @ dod.abs())]
    errs = [e + H8 * x.abs() for e, x in zip(errs, grads)]
    rounded = [scale ** 2 * (dS ** 2 @ kd ** 2).sum(), scale ** 2 * (to_k ** 2 @ qd ** 2).sum(),
               ((P ** 2).transpose(1, 2) @ dod ** 2).sum()]
    return [x.transpose(0, 1) for x in grads], [x.transpose(0, 1) for x in errs], rounded


def reference(torch, q, k, v, do, lens, window, scale):
    parts, at = [], 0
    for n in lens:
        if n:
            parts.append(sequence(torch, *(t[at:at + n] for t in (q, k, v, do)), window, scale))
        at += n
    grads = [torch.cat([p[0][i] for p in parts]) for i in range(3)]
    errs = [torch.cat([p[1][i] for p in parts]) for i in range(3)]
    return grads, errs, [sum(p[2][i] for p in parts) for i in range(3)]


def run(torch, lens, H, Hkv, window, scale, seed):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu = make(torch, lens, H, Hkv, seed)
    plan = g.attention_plan(cu, sum(lens), window=window)
    o, lse = g.attention_packed_fwd(q, k, v, plan, scale=scale)
    got = g.attention_packed_bwd(q, k, v, o, lse, do, plan, scale=scale)
    g.op_check()
    return got, reference(torch, q, k, v, do, lens, window, scale)


@pytest.mark.parametrize("sharp", [1, 8])
@pytest.mark.parametrize("length,count,H,Hkv", [(2, 100, 4, 4), (3, 80, 4, 2), (5, 60, 4, 4), (40, 10, 6, 2),
                                                (300, 5, 4, 4)])
def test_norms(torch, length, count, H, Hkv, sharp):
    """Scores of the usual size and eight times as large, where a row's
    probability sits on one key and dP - D of that key is small."""
    got, (grads, _, rounded) = run(torch, [length] * count, H, Hkv, -1, sharp / math.sqrt(128), length)
    for name, x, want, r in zip(("dq", "dk", "dv"), got, grads, rounded):
        off = float((x.double() - want).norm() / want.norm())
        allowed = 1.25 * RMS * math.sqrt(1 + float(r) / float(want.norm()) ** 2)
        assert off <= allowed, (name, off, allowed)


@pytest.mark.parametrize("sharp", [1, 8])
@pytest.mark.parametrize("lens,H,Hkv,window", [([2] * 200, 1, 1, -1), ([1, 2, 3, 4, 5, 6, 7] * 20, 3, 1, -1),
                                               ([40, 7, 129, 1, 0, 300, 128], 4, 2, -1), ([500, 3, 140], 2, 2, 30),
                                               ([700], 2, 1, -1)])
def test_elements(torch, lens, H, Hkv, window, sharp):
    got, (grads, errs, _) = run(torch, lens, H, Hkv, window, sharp / math.sqrt(128), len(lens))
    for name, x, want, e in zip(("dq", "dk", "dv"), got, grads, errs):
        over = (x.double() - want).abs() / (e + 1e-30)
        assert float(over.max()) <= 1, (name, float(over.max()), int((over > 1).sum()))
