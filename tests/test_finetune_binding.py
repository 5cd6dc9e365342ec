"""What the fine-tuning calls refuse before any device work, and what their
binding does around them, without a GPU."""
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


def test_rows_of_logits_past_what_loops_in_32_bits_reach(g):
    """The last index plus a loop's step has to fit in an int."""
    L = g.lib()
    for M in ((1 << 30) + 1, (1 << 31) - 1):
        policy = L.gpt_op_policy_loss(A, 0, 8, A, None, None, A, A, M, 8, 0.2, 0.2, 0.0, A, A, A, 8, A, None)
        preference = L.gpt_op_preference_loss(A, 0, 8, A, A, 2, None, M, 8, 0.1, 0.0, A, A, A, A, A, 8, A, None)
        assert policy == preference == g.GPT_EINVAL and b"2^30" in L.gpt_last_error()
