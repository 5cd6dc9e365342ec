"""Tensors of another rank than the fine-tuning calls take (B200 only)."""
import pytest

pytestmark = pytest.mark.gpu


def test_ranks():
    import torch
    import gpt_pretraining_step_b200 as g
    n = 64
    t = torch.zeros((n, 2, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 30, n], dtype=torch.int32, device="cuda")
    plan = g.attention_plan(cu, n)
    o, lse = g.attention_packed_fwd(t, t, t, plan)
    other = [t[0, 0], t[:, 0], t[None], t[0, 0, 0], t.view(n, 2, 2, 64)]
    x, y, a = torch.zeros((n, 8), device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"), o.new_zeros(
        n, dtype=torch.float32)
    calls = [lambda b: g.attention_packed_fwd(b, t, t, plan), lambda b: g.attention_packed_fwd(t, b, t, plan),
             lambda b: g.attention_packed_fwd(t, t, b, plan), lambda b: g.attention_packed_fwd(t, t, t, plan, o=b),
             lambda b: g.attention_packed_bwd(b, t, t, o, lse, o, plan),
             lambda b: g.attention_packed_bwd(t, b, t, o, lse, o, plan),
             lambda b: g.attention_packed_bwd(t, t, t, b, lse, o, plan),
             lambda b: g.attention_packed_bwd(t, t, t, o, b.float(), o, plan),
             lambda b: g.attention_packed_bwd(t, t, t, o, lse, b, plan),
             lambda b: g.attention_packed_bwd(t, t, t, o, lse, o, plan, dk=b),
             lambda b: g.policy_loss(b[..., :8] if b.dim() != 2 else b[None], y, a, a, a),
             lambda b: g.policy_loss(x, b.int(), a, a, a), lambda b: g.policy_loss(x, y, a, b.float(), a),
             lambda b: g.preference_loss(x, y, cu, ref_logp=b.float()),
             lambda b: g.preference_loss(x, y, cu, dlogits=b.float()), lambda b: g.attention_plan(b.int()[None], n)]
    for i, call in enumerate(calls):
        for b in other:
            if b.dim() == 0 and i in (10, len(calls) - 1):
                continue    # no slice of it; one offset is a batch without sequences
            with pytest.raises(g.GptError) as e:
                call(b)
            assert e.value.code == g.GPT_EINVAL, i
    g.op_check()
