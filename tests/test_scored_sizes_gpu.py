"""Scored attention at sizes that the dense comparisons of test_scored_gpu.py cannot hold: long block lists, whose
filtering takes many rounds, and a 720p latent, whose tiles are launched as they are (not by length)."""
import math

import numpy as np
import pytest
import torch

from test_scored_gpu import E, FP32, Case, P  # noqa: F401  (the fixture)

FORMS = {
    "clips": dict(clips=5, padding=1, causal=True, prefix=1),
    "tokens": dict(cap=20.0, clips=40, padding=2, shuffled=True),
    "all": dict(cap=15.0, slope=0.2, clips=6, padding=3, causal=True, prefix=2, pos="given"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("hilbert", [64, 128])
@pytest.mark.parametrize("form", list(FORMS))
def test_long_lists(P, form, hilbert):  # noqa: F811
    """Every block selected: lists of 48 or 96 blocks, filtered 32 at a time, some of each 32 hidden."""
    c = Case(P, 16, 16, 24, 2, 64, top_k=96, frac=1.0, top_p=1.0, hilbert=hilbert, seed=70, **FORMS[form])
    v = c.plan.view()
    assert v["n_blocks"][0] == c.N // hilbert and int(v["row_ptr"][1]) == c.N // hilbert > 32
    c.check()
    c.plan.close()


def by_head(c, h, step=512):
    """O, lse, dQ, dK, dV of head h and the bounds of test_scored_gpu.py, `step` queries at a time."""
    N, scale = c.N, 1 / math.sqrt(c.dim)
    q, k, v, do = (x[0, :, h].double() for x in (c.Q, c.K, c.V, c.dO))
    if c.doc is not None:
        pad = (c.doc[0] < 0)[:, None]
        q, k, v, do = (x.masked_fill(pad, 0) for x in (q, k, v, do))
    view = c.plan.view()
    nb, nbmax = view["n_blocks"][0], view["nbmax"]
    off = view["blk_off"][0][:nb + 1].long()
    blk = torch.empty(N, dtype=torch.int64, device="cuda")
    blk[view["perm"][0].long()] = torch.repeat_interleave(torch.arange(nb, device="cuda"), off[1:] - off[:-1])
    ptr = view["row_ptr"][h * nbmax:][:nb + 1].long()
    sel = torch.zeros(nb, nb, dtype=torch.bool, device="cuda")
    rows = torch.repeat_interleave(torch.arange(nb, device="cuda"), ptr[1:] - ptr[:-1])
    sel[rows, view["col_idx"][ptr[0]:ptr[-1]].long()] = True
    p = c.position[0]
    out = {n: torch.zeros(N, c.dim, dtype=torch.float64, device="cuda") for n in ("O", "eO", "dQ", "eQ", "dK", "eK", "dV", "eV")}
    out["lse"] = torch.empty(N, dtype=torch.float64, device="cuda")
    for i in range(0, N, step):
        s = slice(i, i + step)
        x = q[s] @ k.T * scale
        t1 = torch.ones((), device="cuda", dtype=torch.float64)
        if c.cap:
            t = torch.tanh(x / c.cap)
            x, t1 = c.cap * t, 1 - t * t
        if c.slopes is not None:
            x -= float(c.slopes[h]) * (p[s, None] - p).abs()
        seen = sel[blk[s]][:, blk]
        if c.doc is not None:
            seen &= (c.doc[0, s, None] == c.doc[0]) & (c.doc[0] >= 0)
        if c.causal:
            seen &= (p <= p[s, None]) | (p < (c.prefix[0] if c.prefix is not None else -math.inf))
        x.masked_fill_(~seen, -math.inf)
        lse = torch.logsumexp(x, 1)
        w = torch.exp(x - torch.where(lse.isfinite(), lse, 0)[:, None])
        O = w @ v
        wv = w @ v.abs()
        eO = (E + FP32) * wv + E * O.abs()
        ds = w * (do[s] @ v.T - (do[s] * O).sum(1, keepdim=True)) * t1
        eds = (E + FP32) * ds.abs() + w * t1 * ((do[s].abs() * eO).sum(1, keepdim=True) + FP32 * (do[s].abs() @ v.abs().T))
        out["O"][s], out["eO"][s], out["lse"][s] = O, eO, lse
        out["dQ"][s] = ds @ k * scale
        out["eQ"][s] = scale * (eds @ k.abs())
        out["dK"] += ds.T @ q[s] * scale
        out["eK"] += scale * (eds.T @ q[s].abs())
        out["dV"] += w.T @ do[s]
        out["eV"] += (E + FP32) * (w.T @ do[s].abs())
    for n in ("Q", "K", "V"):
        out["e" + n] += E * out["d" + n].abs()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("form", [dict(cap=20.0, slope=0.25),
                                  dict(cap=30.0, slope=0.125, clips=3, padding=1, causal=True, prefix=2)])
def test_a_720p_latent(P, form):  # noqa: F811
    """24 x 48 x 80 tokens: K and V of four heads pass the forward's limit for a launch order by length (160 MB), their
    2880 key tiles the backward's (1184).  One head is compared as a whole."""
    c = Case(P, 24, 48, 80, 4, 128, top_k=16, frac=0.0625, seed=71, **form)
    assert 4 * c.N * c.dim * 4 > 160e6 and 4 * c.N // 128 > 1184
    got = c.run()
    h = int(np.random.default_rng(71).integers(4))
    r = by_head(c, h)
    none = r["lse"] == -math.inf
    lse = got["lse"][0, h].double()
    assert torch.equal(lse == -math.inf, none) and ((lse - r["lse"])[~none].abs() < 1e-4).all()
    for n, e in (("O", "eO"), ("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
        off = (got[n][0, :, h].double() - r[n]).abs()
        assert (off <= r[e] + 1e-30).all(), (n, h, (off - r[e]).max().item())
    c.plan.close()
