"""Range of the scored forward's running-maximum tiles: what O can hold, its sums have to hold."""
import pytest
import torch

from test_scored_gpu import Case, P  # noqa: F401  (the fixture)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [100, 107, 116])
@pytest.mark.parametrize("rise", [5.0, 11.0, 16.0, 40.0])
def test_large_values_under_logits_that_rise_along_the_keys(P, rise, power):  # noqa: F811
    """The later half of the keys has logits `rise` above the first half's (23 powers of two at 16), with values of
    2^power: against the first half's maximum their products pass fp32's largest number, O does not.  O is linear in V:
    over 2^power it has the bounds of power = 0."""
    c = Case(P, 16, 8, 16, 2, 64, seed=80)
    c.Q[..., 0] = 8.0
    c.K[..., 0] = 0.0
    c.K[:, c.N // 2:, :, 0] = rise
    c.plan.update_qkv(c.Q, c.K, c.V * 2.0 ** power)
    O, _ = c.plan.fwd(scored=True)
    c.plan.check()
    for h in range(2):
        ref, err = c.reference(0, h)
        off = (O[0, :, h].double() * 2.0 ** -power - ref["O"]).abs()
        assert (off <= err["O"] + 1e-30).all(), (h, (off - err["O"]).max().item())
    c.plan.close()
