"""Refusals of the fine-tuning calls through the C ABI: every one comes before
any device work, so they are checked without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def g():
    import gpt_pretraining_step_b200 as g
    import os
    if not os.path.exists(g.LIB_PATH):
        from gpt_pretraining_step_b200 import build
        build.build(verbose=False)
    g.lib()
    return g


A = 0x10000   # an aligned address that no refused call reads


def heads(g, data=A, token=256, head=128):
    return g.Heads(data, token, head)


def test_sizes(g):
    L = g.lib()
    for n in (0, 1, 127, 128, 129, 5000):
        tiles = (n + 127) // 128
        assert L.gpt_op_attention_plan_bytes(n) >= 8 * n + 16 * tiles
        # -lse and -D in whole tiles and the fp32 dq
        assert L.gpt_op_attention_packed_bwd_scratch(n, 3) >= 3 * (8 * 128 * tiles + 512 * n)
    assert L.gpt_op_attention_plan_bytes(-1) == 0
    assert L.gpt_op_attention_packed_bwd_scratch(5, 0) == 0 and L.gpt_op_attention_packed_bwd_scratch(-1, 2) == 0
    assert L.gpt_op_policy_loss_scratch(100) >= 1600 and L.gpt_op_policy_loss_scratch(-1) == 0
    assert L.gpt_op_preference_loss_scratch(100, 4) >= 1600 and L.gpt_op_preference_loss_scratch(100, 0) == 0


def test_plan(g):
    L = g.lib()
    for args in [(None, 1, 64, -1, A, None), (A, 1, 64, -1, None, None), (A, -1, 64, -1, A, None),
                 (A, 1, -1, -1, A, None), (A, 1, (1 << 30) + 1, -1, A, None), (A, 1, 64, -1, A + 16, None)]:
        assert L.gpt_op_attention_plan(*args) == g.GPT_EINVAL, args


def test_packed_attention(g):
    L = g.lib()
    ok = dict(q=heads(g), k=heads(g), v=heads(g), o=heads(g), lse=A, n=64, H=2, Hkv=2, scale=0.0, plan=A)

    def fwd(**kw):
        a = dict(ok, **kw)
        return L.gpt_op_attention_packed_fwd(a["q"], a["k"], a["v"], a["o"], a["lse"], a["n"], a["H"], a["Hkv"],
                                             a["scale"], a["plan"], None)

    def bwd(**kw):
        a = dict(ok, dout=heads(g), dq=heads(g), dk=heads(g), dv=heads(g), scratch=A)
        a.update(kw)
        return L.gpt_op_attention_packed_bwd(a["q"], a["k"], a["v"], a["o"], a["lse"], a["dout"], a["dq"], a["dk"],
                                             a["dv"], a["n"], a["H"], a["Hkv"], a["scale"], a["plan"], a["scratch"],
                                             None)

    common = [dict(n=-1), dict(H=0), dict(Hkv=0), dict(H=3, Hkv=2), dict(scale=-1.0), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(plan=None), dict(plan=A + 8), dict(lse=None), dict(q=None),
              dict(k=heads(g, data=None)), dict(q=heads(g, data=A + 8)), dict(v=heads(g, token=257)),
              dict(k=heads(g, head=4)), dict(q=heads(g, token=-256)), dict(n=1 << 30, H=4, Hkv=4)]
    outputs = [dict(token=128), dict(head=64), dict(token=0), dict(token=8, head=8)]   # rows that overlap
    for kw in common + [dict(o=heads(g, **b)) for b in outputs]:
        assert fwd(**kw) == g.GPT_EINVAL, kw
        assert L.gpt_last_error()
    for kw in common + [dict(scratch=None), dict(scratch=A + 128), dict(dout=None)] + [
            {name: heads(g, **b)} for b in outputs for name in ("dq", "dk", "dv")]:
        assert bwd(**kw) == g.GPT_EINVAL, kw
    # nothing to do is not an error, and extents of one take any stride
    assert fwd(n=0) == 0 and bwd(n=0) == 0


def test_losses(g):
    L = g.lib()
    ok = dict(x=A, dtype=g.DTYPE_FP32, ld=64, y=A, M=8, V=50, d=A * 2, ld_d=64, scratch=A)
    common = [dict(dtype=2), dict(dtype=-1), dict(ld=49), dict(ld_d=49), dict(M=-1), dict(V=0), dict(V=(1 << 24) + 1),
              dict(x=None), dict(y=None), dict(scratch=None), dict(scratch=A + 64), dict(x=A + 2),
              dict(d=A, ld_d=72)]

    def policy(old=A, ref=None, adv=A, w=A, lo=0.2, hi=0.2, kl=0.0, stats=A, logp=A, **kw):
        a = dict(ok, **kw)
        return L.gpt_op_policy_loss(a["x"], a["dtype"], a["ld"], a["y"], old, ref, adv, w, a["M"], a["V"], lo, hi, kl,
                                    stats, logp, a["d"], a["ld_d"], a["scratch"], None)

    def preference(cu=A, pairs=2, beta=0.1, smooth=0.0, loss=A, margin=A, seq=A, logp=A, **kw):
        a = dict(ok, **kw)
        return L.gpt_op_preference_loss(a["x"], a["dtype"], a["ld"], a["y"], cu, pairs, None, a["M"], a["V"], beta,
                                        smooth, loss, margin, seq, logp, a["d"], a["ld_d"], a["scratch"], None)

    nan, inf = float("nan"), float("inf")
    for kw in common + [dict(adv=None), dict(w=None), dict(stats=None), dict(logp=None), dict(lo=-0.1), dict(lo=1.1),
                        dict(lo=nan), dict(hi=-0.1), dict(hi=inf), dict(hi=nan), dict(kl=0.1), dict(ref=A, kl=nan)]:
        assert policy(**kw) == g.GPT_EINVAL, kw
    for kw in common + [dict(cu=None), dict(pairs=0), dict(pairs=(1 << 29) + 1), dict(beta=inf), dict(beta=nan),
                        dict(smooth=-0.1), dict(smooth=1.1), dict(smooth=nan), dict(loss=None), dict(margin=None),
                        dict(seq=None), dict(logp=None)]:
        assert preference(**kw) == g.GPT_EINVAL, kw


def test_binding_refuses_host_tensors(g):
    import torch
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    x, y, a = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for call in (lambda: g.attention_plan(cu, 4), lambda: g.policy_loss(x, y, a, a, a),
                 lambda: g.preference_loss(x, y, torch.tensor([0, 2, 4], dtype=torch.int32))):
        with pytest.raises(g.GptError) as e:
            call()
        assert e.value.code == g.GPT_EINVAL
    assert ctypes.sizeof(g.Heads) == 24 and q.stride() == (256, 128, 1)


def test_binding_refuses_what_32_bits_do_not_hold(g):
    """ctypes drops the upper bits of an int argument, so the binding looks first."""
    import torch
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for n in (2 ** 32 + 4, 2 ** 31, -1):
        with pytest.raises(g.GptError, match="n_tokens"):
            g.attention_plan(cu, n)
    assert g.lib().gpt_op_attention_plan(A, (1 << 30) + 1, 64, -1, A, None) == g.GPT_EINVAL
