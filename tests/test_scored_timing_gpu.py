"""Per-kernel timing of a scored forward."""
import pytest

from test_scored_gpu import Case, P  # noqa: F401  (the fixture)


@pytest.mark.gpu
def test_a_scored_forward_is_one_launch_of_the_forward(P):  # noqa: F811
    """The pass over the tiles put off belongs to the forward: milliseconds over launches is the forward's time."""
    c = Case(P, 8, 16, 16, 2, 64, cap=10.0, seed=40)
    c.plan.set_timing(True)
    for _ in range(3):
        c.plan.fwd(scored=True)
    ms, n = c.plan.read_timing()["attn_fwd"]
    assert n == 3 and ms > 0
    c.plan.fwd()
    assert c.plan.read_timing()["attn_fwd"][1] == 1
    c.plan.set_timing(False)
    c.plan.close()
