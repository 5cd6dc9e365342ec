"""Memory of the fine-tuning calls on streams other than its own (B200 only).
What could be overwritten is never used: the tests look at what the allocator
was told."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    import gpt_pretraining_step_b200 as g
    g.lib()
    return t


class Recorded:
    """A tensor that notes the streams it is recorded on."""

    def __init__(self, t):
        self.t, self.streams = t, []

    def record_stream(self, s):
        self.streams.append(s.cuda_stream)
        self.t.record_stream(s)

    def __getattr__(self, name):
        return getattr(self.t, name)


def packed(torch, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn((300, 2, 128), generator=g, device="cuda").bfloat16() for _ in range(4))
    return q, k, v, do, torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")


def test_a_plan_is_kept_for_the_streams_that_read_it(torch):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu = packed(torch)
    plan = g.attention_plan(cu, 300)
    plan.buf = Recorded(plan.buf)
    want = g.attention_packed_fwd(q, k, v, plan)
    assert plan.buf.streams == []          # its own stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # by argument, and as the current stream
    o, lse = g.attention_packed_fwd(q, k, v, plan, stream=side)
    assert plan.buf.streams == [side.cuda_stream]
    g.attention_packed_bwd(q, k, v, o, lse, do, plan, stream=side)
    assert plan.buf.streams == [side.cuda_stream] * 2
    with torch.cuda.stream(side):
        o2, lse2 = g.attention_packed_fwd(q, k, v, plan)
        g.attention_packed_bwd(q, k, v, o2, lse2, do, plan)
        plan.update(cu)
    assert plan.buf.streams == [side.cuda_stream] * 5
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((o, want[0]), (lse, want[1]), (o2, want[0]), (lse2, want[1])):
        assert torch.equal(a, b)
    g.op_check()


def test_entries_out_of_bounds_are_left_out(torch):
    """A plan whose entries have been overwritten: the words that the kernels
    index with are bounded, the error is reported and the calls end."""
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu = packed(torch)
    o, lse = g.attention_packed_fwd(q, k, v, g.attention_plan(cu, 300))
    head, per, tiles = 64, 300, 3         # words before lo, of lo and of hi, tiles of 128
    fwd, bwd = head + 2 * per, head + 2 * per + 2 * tiles
    for at, pair in ((fwd, (1 << 30, 0)), (fwd + 2, (-1, -5)), (fwd + 4, (1, 2)), (fwd, (0, -(1 << 30))),
                     (bwd, (1 << 30, 1)), (bwd + 2, (-3, 1)), (bwd + 4, (1, 1 << 30)), (bwd, (2, 2)), (bwd, (1, 0))):
        plan = g.attention_plan(cu, 300)
        plan.buf[at:at + 2] = torch.tensor(pair, dtype=torch.int32, device="cuda")
        g.attention_packed_fwd(q, k, v, plan)
        g.attention_packed_bwd(q, k, v, o, lse, do, plan)
        with pytest.raises(g.GptError):
            g.op_check()
    # sizes
    for at, value in ((0, 1 << 30), (0, -7), (1, 1 << 30), (1, -1), (2, 1 << 30), (2, -1)):
        plan = g.attention_plan(cu, 300)
        plan.buf[at] = value
        plan.buf[fwd + 6 + 6:] = 0
        g.attention_packed_fwd(q, k, v, plan)
        g.attention_packed_bwd(q, k, v, o, lse, do, plan)
    g.op_check()
    plan = g.attention_plan(cu, 300)
    o2, lse2 = g.attention_packed_fwd(q, k, v, plan)
    g.op_check()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
