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
