"""Losses on logits of more than 2^31 elements (B200 only): the first and the last
rows against 64 bits, with the bounds of test_gpu_losses."""
import pytest

from test_gpu_losses import check_grad, check_lp, exact_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def test_offsets_past_32_bits(torch):
    import gpt_pretraining_step_b200 as gpt
    M, V, pad = 70000, 32768, 100
    assert M * V > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((M, V), dtype=torch.bfloat16, device="cuda").normal_(0, 2, generator=gen)
    y = torch.randint(0, V, (M,), generator=gen, device="cuda").to(torch.int32)
    adv, w = torch.randn(M, generator=gen, device="cuda"), torch.rand(M, generator=gen, device="cuda") / M
    stats, logp, d = gpt.policy_loss(x, y, None, adv, w)
    ends = torch.cat([torch.arange(8), torch.arange(M - pad - 8, M)]).cuda()
    seen, lp, p, hot = exact_rows(torch, x[ends], y[ends])
    check_lp(torch, logp[ends], lp)
    g = (-adv * w).double()[ends]
    check_grad(torch, d[ends], seen, g, g.abs(), p, hot)
    assert abs(stats[0].double() + (adv.double() * w.double()).sum()) <= 2e-5 * (adv.abs() * w).sum()
    del d
    cu = torch.tensor([0, 40, 35000, 60000, M - pad], dtype=torch.int32, device="cuda")
    loss, margin, seq, logp2, d = gpt.preference_loss(x, y, cu, beta=0.001, dlogits=x)
    gpt.op_check()
    assert d is x and torch.equal(logp2[:M - pad], logp[:M - pad]) and (logp2[M - pad:] == 0).all()
    sums = torch.stack([logp[a:b].double().sum() for a, b in zip(cu[:-1].tolist(), cu[1:].tolist())])
    # each log-probability is rounded to fp32 (2^-24 of about 13), the sum again
    assert ((seq.double() - sums).abs() <= 2.0 ** -23 * (sums.abs() + 13.0 * (cu[1:] - cu[:-1]))).all()
    z = 0.001 * (seq[0::2] - seq[1::2]).double()
    assert (margin.double() - z).abs().max() <= 2.0 ** -20 * 0.001 * sums.abs().max()
    g = torch.where(ends < 40, 1.0, -1.0) * (-0.0005 * torch.sigmoid(-z))[torch.where(ends < 40, 0, 1)]
    counted = ends < M - pad
    check_grad(torch, d[ends][counted], seen[counted], g[counted], 2 * g[counted].abs(), p[counted], hot[counted])
