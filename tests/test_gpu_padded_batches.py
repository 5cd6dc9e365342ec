"""Batches padded to a fixed capacity: the rows past the last sequence of the
outputs, whatever the inputs hold there (B200 only).

A step multiplies whole buffers: a gradient by the logits meets the hidden
states of every row in the lm_head's gradient.  So what a call allocates itself
holds zeros there; a buffer that the caller gives keeps what it held, unless the
call is told to clear those rows.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


def dirty(torch, *shape, dtype):
    """Leaves a freed block full of NaN for the next tensor of this size."""
    torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def preference_batch(torch, dtype, V, ld, lens, pad, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = sum(lens)
    M = total + pad
    buf = torch.randn((M, ld), generator=g, device="cuda").to(dtype)
    x = buf[:, :V]
    y = torch.randint(0, V, (M,), generator=g, device="cuda").to(torch.int32)
    y[total:] = -1
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return x, y, torch.tensor(cu, dtype=torch.int32, device="cuda"), total


SHAPES = [("bfloat16", 1000, 1000, [20, 13, 0, 40], 55), ("float32", 1001, 1003, [3, 4], 1),
          ("bfloat16", 40000, 40000, [5, 6], 300), ("float32", 77, 77, [0, 0], 9), ("bfloat16", 5003, 5003, [7, 9], 0)]


@pytest.mark.parametrize("dtype,V,ld,lens,pad", SHAPES)
@pytest.mark.parametrize("fill", ["finite", "nan"])
def test_preference(torch, dtype, V, ld, lens, pad, fill):
    import gpt_pretraining_step_b200 as gpt
    dt = getattr(torch, dtype)
    x, y, cu, total = preference_batch(torch, dt, V, ld, lens, pad)
    if fill == "nan":
        x[total:] = float("nan")
    M = x.shape[0]
    want = gpt.preference_loss(x[:total], y[:total], cu) if total else None

    def same(out):
        assert (out[4][total:] == 0).all() and (out[3][total:] == 0).all()
        for i in range(3) if want else ():
            assert torch.equal(out[i], want[i])
        if want:
            assert torch.equal(out[3][:total], want[3]) and torch.equal(out[4][:total], want[4])

    dirty(torch, M, V, dtype=dt)
    dirty(torch, M, dtype=torch.float32)
    same(gpt.preference_loss(x, y, cu))
    # a given gradient keeps its rows there, unless they are to be cleared; its log-probabilities are new
    d = torch.full((M, V), 7.0, dtype=dt, device="cuda")
    out = gpt.preference_loss(x, y, cu, dlogits=d)
    assert (d[total:] == 7.0).all() and (out[3][total:] == 0).all()
    same(gpt.preference_loss(x, y, cu, dlogits=d, clear_past=True))
    keep = x[total:].clone()

    def copy():   # with the same strides: rows aligned otherwise add up in another order
        return torch.empty((M, ld), dtype=dt, device="cuda")[:, :V].copy_(x)

    inplace = copy()
    out = gpt.preference_loss(inplace, y, cu, dlogits=inplace)
    assert torch.equal(out[4][total:].nan_to_num(5.0), keep.nan_to_num(5.0))
    inplace = copy()
    same(gpt.preference_loss(inplace, y, cu, dlogits=inplace, clear_past=True))
    out = gpt.preference_loss(x, y, cu, grad=False)
    assert out[4] is None and (out[3][total:] == 0).all()
    gpt.op_check()


def test_preference_replayed_with_other_lengths(torch):
    """A captured call clears what the offsets of each replay leave."""
    import gpt_pretraining_step_b200 as gpt
    x, y, cu, _ = preference_batch(torch, torch.bfloat16, 3000, 3000, [20, 20], 24)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpt.preference_loss(x, y, cu)
    for edges in ([0, 20, 40], [0, 5, 64], [0, 1, 3], [0, 10, 33]):
        cu.copy_(torch.tensor(edges, dtype=torch.int32))
        y.copy_(torch.randint(0, 3000, (64,), device="cuda"))
        out[4].fill_(float("nan"))
        graph.replay()
        gpt.op_check()
        want = gpt.preference_loss(x[:edges[-1]], y[:edges[-1]], cu)
        assert torch.equal(out[4][:edges[-1]], want[4]) and (out[4][edges[-1]:] == 0).all()
        assert (out[3][edges[-1]:] == 0).all()


def test_preference_bad_offsets_clear_nothing(torch):
    import gpt_pretraining_step_b200 as gpt
    x, y, _, _ = preference_batch(torch, torch.float32, 50, 50, [3, 3], 4)
    d = torch.full_like(x, 7.0)
    gpt.preference_loss(x, y, torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda"), dlogits=d, clear_past=True)
    with pytest.raises(gpt.GptError) as e:
        gpt.op_check()
    assert e.value.code == gpt.GPT_ERANGE and (d == 7.0).all()


def attention_batch(torch, lens, pad, H, Hkv, fill, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = sum(lens)
    x = torch.randn((total + pad, 2 * H + 2 * Hkv, 128), generator=g, device="cuda").bfloat16()
    x[total:] = fill
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return (*x.split([H, Hkv, Hkv, H], 1), torch.tensor(cu, dtype=torch.int32, device="cuda"), total)


@pytest.mark.parametrize("lens,pad", [([100, 60], 1), ([100, 28], 128), ([100, 27], 700), ([1], 3000), ([], 150),
                                      ([0, 0], 10), ([300, 84], 0), ([256], 40), ([40] * 60, 2700)])
@pytest.mark.parametrize("H,Hkv", [(3, 1), (4, 4)])
def test_attention(torch, lens, pad, H, Hkv):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu, total = attention_batch(torch, lens, pad, H, Hkv, float("nan"))
    n = total + pad
    plan = g.attention_plan(cu, n)

    def marked(*shape, dtype=torch.bfloat16):
        return torch.full(shape, 7.0, dtype=dtype, device="cuda")

    def forward(**kw):
        return g.attention_packed_fwd(q, k, v, plan, **kw)

    # given: rows past the sequences stay
    o, lse = forward(o=marked(n, H, 128), lse=marked(H, n, dtype=torch.float32))
    assert (o[total:] == 7.0).all() and (lse[:, total:] == 7.0).all()
    grads = g.attention_packed_bwd(q, k, v, o, lse, do, plan, dq=marked(n, H, 128), dk=marked(n, Hkv, 128),
                                   dv=marked(n, Hkv, 128))
    assert all((t[total:] == 7.0).all() for t in grads)
    # new: zeros there, the others' rows the same
    for shape, dt in (((n, H, 128), torch.bfloat16), ((H, n), torch.float32), ((n, Hkv, 128), torch.bfloat16)):
        dirty(torch, *shape, dtype=dt)
        dirty(torch, *shape, dtype=dt)
    o2, lse2 = forward()
    new = g.attention_packed_bwd(q, k, v, o2, lse2, do, plan)
    assert (o2[total:] == 0).all() and (lse2[:, total:] == 0).all()
    assert torch.equal(o2[:total], o[:total]) and torch.equal(lse2[:, :total], lse[:, :total])
    assert all((t[total:] == 0).all() for t in new)
    assert torch.equal(new[1][:total], grads[1][:total]) and torch.equal(new[2][:total], grads[2][:total])
    # one given, the others new
    o3, lse3 = forward(o=marked(n, H, 128))
    assert (o3[total:] == 7.0).all() and (lse3[:, total:] == 0).all()
    o4, lse4 = forward(lse=marked(H, n, dtype=torch.float32))
    assert (o4[total:] == 0).all() and (lse4[:, total:] == 7.0).all()
    for i, name in enumerate(("dq", "dk", "dv")):
        mixed = g.attention_packed_bwd(q, k, v, o, lse, do, plan, **{name: marked(n, Hkv if i else H, 128)})
        for j, t in enumerate(mixed):
            assert (t[total:] == (7.0 if i == j else 0.0)).all(), (name, j)
    # given ones, cleared on request; in slices of a wider buffer, whose other columns stay
    wide = marked(n, 2 * H + 2 * Hkv + 1, 128)
    parts = wide.split([H, H, Hkv, Hkv, 1], 1)
    o5, lse5 = forward(o=parts[0], lse=marked(H, n, dtype=torch.float32), clear_past=True)
    g.attention_packed_bwd(q, k, v, o, lse, do, plan, dq=parts[1], dk=parts[2], dv=parts[3], clear_past=True)
    assert (wide[total:, :-1] == 0).all() and (wide[:, -1] == 7.0).all() and (lse5[:, total:] == 0).all()
    assert torch.equal(o5[:total], o[:total]) and torch.equal(parts[3][:total], grads[2][:total])
    g.op_check()


def test_attention_replayed_with_other_lengths(torch):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu, _ = attention_batch(torch, [100, 200], 400, 2, 1, 1.0)
    n = 700
    plan = g.attention_plan(cu, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.update(cu)
        o, lse = g.attention_packed_fwd(q, k, v, plan)
        grads = g.attention_packed_bwd(q, k, v, o, lse, do, plan)
    for edges in ([0, 100, 300], [0, 1, 700], [0, 0, 0], [0, 5, 129], [0, 300, 640]):
        cu.copy_(torch.tensor(edges, dtype=torch.int32))
        for t in (o, lse, *grads):
            t.fill_(float("nan"))
        graph.replay()
        g.op_check()
        at = edges[-1]
        for t in (o[at:], lse[:, at:], *(t[at:] for t in grads)):
            assert (t == 0).all(), edges
        assert o[:at].isfinite().all() and lse[:, :at].isfinite().all() and all(t[:at].isfinite().all() for t in grads)


def test_a_whole_step_of_a_padded_batch(torch):
    """Packed attention, projections and the preference loss in new buffers:
    weight gradients of a padded batch, whose pad rows hold anything, are those of
    the batch without padding."""
    import gpt_pretraining_step_b200 as gpt
    g = torch.Generator(device="cuda").manual_seed(1)
    d, V, lens, pad = 256, 500, [30, 50, 7, 60], 200
    total = sum(lens)
    w = [(torch.randn(s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16() for s in ((d, 512), (256, d), (d, V))]
    cu = torch.tensor([0, 30, 80, 87, 147], dtype=torch.int32, device="cuda")
    x = torch.randn((total + pad, d), generator=g, device="cuda").bfloat16()
    y = torch.randint(0, V, (total + pad,), generator=g, device="cuda").to(torch.int32)

    def step(x, y):
        n = x.shape[0]
        plan = gpt.attention_plan(cu, n)
        q, k, v = (x @ w[0]).view(n, 4, 128).split([2, 1, 1], 1)
        o, lse = gpt.attention_packed_fwd(q, k, v, plan)
        h = o.view(n, 256) @ w[1]
        dl = gpt.preference_loss(h @ w[2], y, cu)[4]
        dh = dl @ w[2].t()
        dqkv = torch.empty((n, 4, 128), dtype=torch.bfloat16, device="cuda")
        new = gpt.attention_packed_bwd(q, k, v, o, lse, (dh @ w[1].t()).view(n, 2, 128), plan)
        torch.cat(new, 1, out=dqkv)
        return [x.t().float() @ dqkv.view(n, 512).float(), o.view(n, 256).t().float() @ dh.float(),
                h.t().float() @ dl.float()]

    for t in (x[:total], x):       # leave NaN where the new tensors will be
        for width in (256, 512, d, V):
            dirty(torch, t.shape[0], width, dtype=torch.bfloat16)
    padded, whole = step(x, y), step(x[:total], y[:total])
    gpt.op_check()
    for a, b in zip(padded, whole):
        # products in bf16 of other sizes may add up in another order: three roundings of 2^-8 in a row, of the largest
        assert (a - b).abs().max() <= 3 * 2.0 ** -8 * b.abs().max()
