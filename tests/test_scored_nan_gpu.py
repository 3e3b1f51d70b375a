"""NaN in visible tokens of the scored attention: what sees it is NaN, as the definition says, and nothing else changes.

Which form of tanh a warp takes goes by its largest score, so every case runs with scores below the cap (the polynomial)
and above it (the logistic).  A tile with a NaN row is computed a second time with a running maximum, so the rows beside
it are held to the definition's bounds (test_scored_gpu.py), not to the same bits.
"""
import math

import pytest
import torch

from test_attn_ckpt_gpu import definition
from test_scored_gpu import Case

LEVELS = {"below the cap": dict(cap=60.0, gain=1.0), "above the cap": dict(cap=2.0, gain=2.0)}
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
@pytest.mark.parametrize("level", list(LEVELS))
@pytest.mark.parametrize("which", ["query", "key"])
def test_a_nan_under_a_cap(P, which, level, mask):
    c = Case(P, **GRID, **LEVELS[level], **MASKS[mask], seed=31)
    assert check_forward(c) == 0
    n = inside(c)
    (c.Q if which == "query" else c.K)[0, n, :, 5] = math.nan
    c.plan.update_qkv(c.Q, c.K, c.V)
    hit = check_forward(c)
    assert hit == 2 if which == "query" else hit >= 2
    c.plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("level", list(LEVELS))
def test_scores_of_both_signs_of_infinity_under_a_cap(P, level):
    """tanh of an infinite score is 1 in size: such scores are ordinary ones."""
    c = Case(P, **GRID, **LEVELS[level], seed=32)
    big = torch.zeros(c.dim, device="cuda").bfloat16()
    big[5] = 2.0 ** 100
    c.Q[0, 700] = big                # scores of 2^100 K[k][5]: past the cap, finite
    c.K[0, 900] = big * -2.0 ** 20   # against that query -2^220: an infinity in fp32
    c.plan.update_qkv(c.Q, c.K, c.V)
    assert check_forward(c) == 0
    c.plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("level", list(LEVELS))
def test_a_nan_in_a_checkpoint(P, level, mask):
    """A group of a query's 8-bit values that reads back as NaN, under the healthy forward's log-sum-exp: dV of the keys
    that this query sees and its own dQ are NaN, every other dV and dQ is as if it were not there."""
    c = Case(P, **GRID, **LEVELS[level], **MASKS[mask], seed=33)
    O, lse = c.plan.fwd(scored=True)
    kept = c.plan.save(c.Q, c.K, c.V, O, lse)
    vals = [P.prism_ckpt_unpack(k) for k in (kept.Q, kept.K, kept.V, kept.O)]
    n = inside(c)
    kept.Q.scales[n] = 255
    dQ, _, dV = c.plan.bwd_ckpt(kept, c.dO, scored=True)
    torch.cuda.synchronize()
    c.plan.check()
    clean = c.dO.clone()
    clean[0, n] = 0                  # the query's part of dV
    rest = torch.arange(c.N, device="cuda") != n
    for h in range(c.heads):
        (wq, eq), _, _ = definition(c, 0, h, vals, lse, True)
        keep, c.dO = c.dO, clean
        _, _, (wv, ev) = definition(c, 0, h, vals, lse, True)
        c.dO = keep
        sees = c.allowed(0, h)[n]
        assert dQ[0, n, h].isnan().all() and torch.equal(dV[0, :, h].isnan().all(1), sees)
        assert ((dQ[0, :, h].double() - wq).abs() <= eq + 1e-30)[rest].all()
        assert ((dV[0, :, h].double() - wv).abs() <= ev + 1e-30)[~sees].all()
    c.plan.close()


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
