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
