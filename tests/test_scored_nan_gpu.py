"""NaN in visible tokens of the scored attention: what sees it is NaN, as the definition says, and nothing else changes.

A tile with a NaN row is computed a second time with a running maximum, so the rows beside
it are held to the definition's bounds (test_scored_gpu.py), not to the same bits.
"""
import math

import pytest
import torch

from test_scored_gpu import Case

MASKS = {"none": dict(), "causal": dict(causal=True, prefix=1), "tokens": dict(clips=3, padding=1, shuffled=True),
         "bias": dict(slope=0.3, clips=2)}
GRID = dict(T=16, H=8, W=16, heads=2, dim=64)


@pytest.fixture(scope="module")
def P():
    from dynamic_block_sparse_zone_b200 import build as b
    b.build()
    import dynamic_block_sparse_zone_b200 as P
    P.load_library()
    return P


def inside(c):
    """A token that sees some of the keys and is seen by some of the queries, in every head."""
    a = [c.allowed(0, h) for h in range(c.heads)]
    ok = torch.stack([s.any(1) & s.any(0) & ~s.all(1) for s in a]).all(0)
    ok[:700] = False
    return int(ok.nonzero()[0])


def check_forward(c):
    O, lse = c.plan.fwd(scored=True)
    torch.cuda.synchronize()
    c.plan.check()
    hit = 0
    for h in range(c.heads):
        ref, err = c.reference(0, h)
        nan = ref["lse"].isnan()
        hit += int(nan.sum())
        assert torch.equal(lse[0, h].isnan(), nan) and torch.equal(O[0, :, h].isnan().all(1), nan)
        assert torch.equal(lse[0, h] == -math.inf, ref["lse"] == -math.inf)
        some = ~nan & (ref["lse"] != -math.inf)
        assert ((lse[0, h].double() - ref["lse"])[some].abs() < 1e-4).all()
        off = (O[0, :, h].double() - ref["O"])[~nan].abs()
        assert (off <= err["O"][~nan] + 1e-30).all(), (h, off.max().item())
    return hit


@pytest.mark.gpu
@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("which", ["query", "key"])
def test_a_nan_without_a_cap(P, which, mask):
    """A row whose every visible score is NaN is no row without a key, however its groups of keys are masked."""
    c = Case(P, **GRID, **MASKS[mask], seed=34)
    assert check_forward(c) == 0
    n = inside(c)
    (c.Q if which == "query" else c.K)[0, n, :, 5] = math.nan
    c.plan.update_qkv(c.Q, c.K, c.V)
    hit = check_forward(c)
    assert hit == 2 if which == "query" else hit >= 2
    c.plan.close()
