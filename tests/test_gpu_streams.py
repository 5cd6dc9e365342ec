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


def loss_inputs(torch):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((40, 3000), generator=g, device="cuda").bfloat16()
    y = torch.randint(0, 3000, (40,), generator=g, device="cuda").to(torch.int32)
    return x, y, torch.randn(40, device="cuda"), torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")


def home(torch, t):
    """The stream whose pool a tensor's memory is from."""
    at = t.untyped_storage().data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


def test_new_memory_is_of_the_stream_that_the_call_runs_on(torch):
    """A block of another stream's pool may still be in use there."""
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu = packed(torch)
    x, y, a, pairs = loss_inputs(torch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def calls(stream):
        plan = g.attention_plan(cu, 300, stream=stream)
        o, lse = g.attention_packed_fwd(q, k, v, plan, stream=stream)
        grads = g.attention_packed_bwd(q, k, v, o, lse, do, plan, stream=stream)
        return [plan.buf, o, lse, *grads, *g.policy_loss(x, y, None, a, a, stream=stream),
                *g.preference_loss(x, y, pairs, stream=stream)]

    here, there = calls(None), calls(side)
    assert all(home(torch, t) == torch.cuda.current_stream().cuda_stream for t in here)
    assert all(home(torch, t) == side.cuda_stream for t in there)
    assert torch.cuda.current_stream().cuda_stream != side.cuda_stream
    torch.cuda.current_stream().wait_stream(side)
    for i, (s, t) in enumerate(zip(here, there)):
        assert i in (0, 3) or torch.equal(s, t), i      # a plan's order of equal entries and dq's sums vary
    g.op_check()


def test_every_tensor_of_a_call_is_recorded_on_both_streams(torch, monkeypatch):
    import gpt_pretraining_step_b200 as g
    q, k, v, do, cu = packed(torch)
    x, y, a, pairs = loss_inputs(torch)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(here)
    noted = {}

    def note(t, s):
        noted.setdefault(t.data_ptr(), set()).add(s.cuda_stream)
        plain(t, s)

    plain = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", note)
    plan = g.attention_plan(cu, 300, stream=side)
    o, lse = g.attention_packed_fwd(q, k, v, plan, stream=side)
    grads = g.attention_packed_bwd(q, k, v, o, lse, do, plan, stream=side)
    out = [*g.policy_loss(x, y, a, a, a, ref_logp=a, stream=side), *g.preference_loss(x, y, pairs, stream=side)]
    both = {side.cuda_stream, here.cuda_stream}
    for t in [q, k, v, do, cu, o, lse, *grads, x, y, a, pairs, *out]:
        assert noted[t.data_ptr()] == both
    torch.cuda.synchronize()
    # nothing is recorded where there is one stream alone
    noted.clear()
    plan = g.attention_plan(cu, 300)
    g.attention_packed_fwd(q, k, v, plan)
    g.policy_loss(x, y, a, a, a)
    assert not noted
    g.op_check()
