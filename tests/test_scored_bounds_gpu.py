"""Scored attention against the definition in 64 bits, with bounds close enough to tell the kernel's choices apart: P goes to
the tensor cores as two bf16 numbers, and Delta is formed from O before its rounding.  (The bounds of test_scored_gpu.py
also hold for a kernel that rounds P once and forms Delta from the rounded O.)

Queries have eight channels that are not zero, so that a score has eight terms.  First order, u = 2^-23 for an fp32
operation (half of it for a rounded one; the tensor cores truncate), A = scale sum |q||k|:
  logit:  eX = 9 u A + 4 u (|x| + |bias|) + 4e-7 cap                 (products, log2 units and bias, the tanh fit)
  P:      relative d = eX + 4 u                                      (exp2)
  O:      eO = sum P d |v| + |O| sum P d + (2^-15 + 2 n u) sum P|v|  (hi + lo keep 15 bits; n keys, two products each)
          and the returned O lies between the bf16 numbers next to O - eO and O + eO: half a step, wherever O is
  Delta:  eD = sum |dO| (2^-16 |O| + eO) + 65 u sum |dO O|           (what the second bf16 number of O leaves)
  dS:     e |dS| + |dS| (d + sum P d + 4 u) + P t' (eD + 65 u sum |dO||v|) + 2^-20 P |dP - Delta|  (t' = 1 - tanh^2)
  dQ, dK: their products' sums, e of themselves, and (n + 1) u of the sums' magnitudes
with e = 2^-8, half a step of bf16.  The tests also compute what the coarser choices would give and want it refused.
"""
import math

import pytest
import torch

from test_scored_gpu import Case, P  # noqa: F401  (the fixture)

E, U = 2.0 ** -8, 2.0 ** -23
FORMS = {
    "plain": dict(),
    "cap": dict(cap=8.0),
    "past the cap": dict(cap=1.0),
    "bias": dict(slope=0.7),
    "masks": dict(cap=20.0, slope=0.3, clips=2, padding=1, causal=True, prefix=1),
    "tokens": dict(clips=3, padding=1, shuffled=True),
}


def few_channels(c):
    c.Q[..., 8:] = 0
    c.plan.update_qkv(c.Q, c.K, c.V)
    return c


def bounds(c, h):
    """The definition's tensors of head h and the bounds above, and the coarser choices' results."""
    q, k, v, do = (x[0, :, h].double() for x in (c.Q, c.K, c.V, c.dO))
    if c.doc is not None:
        pad = (c.doc[0] < 0)[:, None]
        q, k, v, do = (x.masked_fill(pad, 0) for x in (q, k, v, do))
    scale = 1 / math.sqrt(c.dim)
    x = q @ k.T * scale
    eX = 9 * U * scale * (q.abs() @ k.abs().T) + 4 * U * x.abs()
    t1 = torch.ones_like(x)
    if c.cap:
        t = torch.tanh(x / c.cap)
        x, t1 = c.cap * t, 1 - t * t
        eX = eX + 4e-7 * c.cap
    if c.slopes is not None:
        p = c.position[0]
        bias = float(c.slopes[h]) * (p[:, None] - p).abs()
        x, eX = x - bias, eX + 4 * U * bias
    seen = c.allowed(0, h)
    x = x.masked_fill(~seen, -math.inf)
    n = seen.sum(1, keepdim=True).double()
    lse = torch.logsumexp(x, 1, keepdim=True)
    lse0 = torch.where(lse.isfinite(), lse, 0)
    w = torch.exp(x - lse0)
    d = (eX + 4 * U).masked_fill(~seen, 0)
    D = (w * d).sum(1, keepdim=True)
    O = w @ v
    eO = (w * d) @ v.abs() + O.abs() * D + (2.0 ** -15 + 2 * n * U) * (w @ v.abs())
    once = torch.exp(x).bfloat16().double()  # P rounded to one bf16 number
    O_once = (once @ v / torch.exp(lse0)).bfloat16().double()
    dP = do @ v.T
    Delta = (do * O).sum(1, keepdim=True)
    ds = w * (dP - Delta) * t1
    eD = (do.abs() * (2.0 ** -16 * O.abs() + eO)).sum(1, keepdim=True) + 65 * U * (do * O).abs().sum(1, keepdim=True)
    eds = (E + d + D + 4 * U) * ds.abs() + w * t1 * (eD + 65 * U * (do.abs() @ v.abs().T)) + 2.0 ** -20 * w * (dP - Delta).abs()
    dQ, dK = ds @ k * scale, ds.T @ q * scale
    nk = seen.sum(0)[:, None].double()
    eQ = scale * (eds @ k.abs() + (n + 1) * U * (ds.abs() @ k.abs())) + E * dQ.abs()
    eK = scale * (eds.T @ q.abs() + (nk + 1) * U * (ds.abs().T @ q.abs())) + E * dK.abs()
    rounded = (do * O.bfloat16().double()).sum(1, keepdim=True)
    dQ_rounded = (w * (dP - rounded) * t1) @ k * scale
    return dict(O=O, eO=eO, O_once=O_once, dQ=dQ, eQ=eQ, dQ_rounded=dQ_rounded, dK=dK, eK=eK)


def between(got, want, err):
    return (got >= (want - err).bfloat16().double()) & (got <= (want + err).bfloat16().double())


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", list(FORMS))
def test_o_is_rounded_once(P, form, dim):  # noqa: F811
    c = few_channels(Case(P, 16, 8, 8, 2, dim, gain=3.0, top_p=1.0, frac=0.0, seed=60, **FORMS[form]))
    O, _ = c.plan.fwd(scored=True)
    c.plan.check()
    for h in range(2):
        r = bounds(c, h)
        ok = between(O[0, :, h].double(), r["O"], r["eO"])
        assert ok.all(), (h, int((~ok).sum()))
        assert not between(r["O_once"], r["O"], r["eO"]).all()
    c.plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("form", list(FORMS))
def test_o_is_rounded_once_with_a_running_maximum(P, form):  # noqa: F811
    """Values of 2^116 under exponentials of up to 2^13 and more: tiles whose products leave fp32's range are done again
    (O is linear in V; a power of two rounds nothing)."""
    c = few_channels(Case(P, 16, 8, 8, 2, 64, gain=3.0, top_p=1.0, frac=0.0, seed=61, **FORMS[form]))
    c.plan.update_qkv(c.Q, c.K, c.V * 2.0 ** 116)
    O, _ = c.plan.fwd(scored=True)
    c.plan.check()
    for h in range(2):
        r = bounds(c, h)
        ok = between(O[0, :, h].double() * 2.0 ** -116, r["O"], r["eO"])
        assert ok.all(), (h, int((~ok).sum()))
    c.plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", ["plain", "cap", "bias"])
def test_delta_is_formed_from_o_before_its_rounding(P, form, dim):  # noqa: F811
    """Documents of four tokens: where one key has most of the weight, dP and Delta nearly cancel."""
    c = few_channels(Case(P, 8, 8, 8, 2, dim, gain=3.0, top_p=1.0, frac=0.0, seed=62, **FORMS[form]))
    c.doc = (torch.arange(c.N, device="cuda") // 4).int()[None]
    c.plan.set_score(cap=c.cap, slopes=c.slopes, doc=c.doc)
    O, _ = c.plan.fwd(scored=True)
    dQ, dK, _ = c.plan.bwd(O, c.dO, scored=True)
    torch.cuda.synchronize()
    c.plan.check()
    for h in range(2):
        r = bounds(c, h)
        assert ((dQ[0, :, h].double() - r["dQ"]).abs() <= r["eQ"] + 1e-30).all(), h
        assert ((dK[0, :, h].double() - r["dK"]).abs() <= r["eK"] + 1e-30).all(), h
        assert not ((r["dQ_rounded"] - r["dQ"]).abs() <= r["eQ"] + 1e-30).all()
    c.plan.close()
