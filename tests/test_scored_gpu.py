"""Scored attention (cap, distance bias, documents, padding, causal with a prefix)
against the definition in 64 bits over the plan's own selection.

Bounds, element by element (e = 2^-8, half a step of bf16; first order in e):
the kernel's P and dS are rounded to bf16 before their products, sums are fp32,
outputs are rounded to bf16, so
  |O err|  <= e sum_k P|v| + e |O|
  |dV err| <= e sum_q P|dO| + e |dV|
  |dS err| <= e |dS| + P (1 - t^2) sum_d |dO_d| |O_d err|     (Delta is formed from the rounded O)
  |dQ err| <= scale sum_k |dS err| |k| + e |dQ|,  |dK err| likewise over q.
What fp32 adds (exp2 and log2 units, the tanh fit's 4e-7 cap, fp32 sums of up to a
few thousand terms) is covered by FP32 = 2^-12 of the same sums.
"""
import math

import numpy as np
import pytest
import torch

E = 2.0 ** -8
FP32 = 2.0 ** -12


@pytest.fixture(scope="module")
def P():
    from dynamic_block_sparse_zone_b200 import build as b
    b.build()
    import dynamic_block_sparse_zone_b200 as P
    P.load_library()
    return P


SHAPES = [(a, b, c) for v in (64, 128, 256) for a in (2, 4, 8) for b in (2, 4, 8) for c in (2, 4, 8) if a * b * c == v]


class Case:
    """A plan on random inputs with random block shapes, its selection as a dense mask, and a score."""

    def __init__(self, P, T, H, W, heads, dim, top_k=3, frac=0.5, batch=1, seed=0, gain=1.5, hilbert=0, cap=0.0, slope=0.0,
                 clips=0, padding=0, causal=False, prefix=None, shuffled=False, pos="frames", top_p=0.9):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rs = np.random.default_rng(seed)
        self.P, self.N, self.heads, self.dim, self.batch, self.cap = P, T * H * W, heads, dim, batch, cap
        N = self.N
        self.Q, self.K, self.V, self.dO = ((s * torch.randn(batch, N, heads, dim, generator=g, device="cuda")).bfloat16()
                                           for s in (gain, gain, 1.0, 1.0))
        self.plan = P.PrismPlan(P.Params(batch=batch, T=T, H=H, W=W, heads=heads, head_dim=dim, top_k=top_k, top_p=top_p,
                                         max_frac=frac, hilbert_block=hilbert))
        if hilbert:
            self.plan.build(self.Q, self.K, self.V, None)
        else:
            shape = rs.integers(0, len(SHAPES), (batch, N // 512)).astype(np.int32)
            self.plan.build_with_zones(self.Q, self.K, self.V, np.vectorize(lambda i: int(np.prod(SHAPES[i])))(shape), shape)
        # documents are runs of frames, or of single tokens (shuffled: any token anywhere)
        frame = torch.arange(N, device="cuda") // (H * W)
        self.doc = self.pos = self.slopes = self.prefix = None
        if clips or padding:
            if shuffled:
                doc = torch.randint(0, max(clips, 1), (batch, N), generator=g, device="cuda")
                doc[torch.rand(batch, N, generator=g, device="cuda") < padding / T] = -5
            else:
                cut = np.sort(rs.choice(np.arange(1, max(2, T - padding)), max(clips, 1) - 1, replace=False)) if clips > 1 else []
                doc = torch.bucketize(frame, torch.tensor(np.asarray(cut, dtype=np.int64), device="cuda"), right=True)
                doc = doc[None].expand(batch, N).clone()
                doc[:, frame >= T - padding] = -1
            self.doc = doc.int()
        if pos == "given":
            self.pos = (torch.randint(0, 6, (batch, N), generator=g, device="cuda") * 0.5 - 1).float()
        self.position = self.pos.double() if self.pos is not None else frame.double()[None].expand(batch, N)
        if slope:
            self.slopes = slope * 0.5 ** torch.arange(heads, device="cuda").float()
        self.causal = causal
        if prefix is not None:
            self.prefix = torch.full((batch,), float(prefix), device="cuda")
        self.plan.set_score(cap=cap, slopes=self.slopes, pos=self.pos, doc=self.doc, causal=causal, prefix=self.prefix)

    def allowed(self, b, h):
        v, N = self.plan.view(), self.N
        nb, nbmax = v["n_blocks"][b], v["nbmax"]
        blk = torch.empty(N, dtype=torch.int64, device="cuda")
        off = v["blk_off"][b][:nb + 1].long()
        blk[v["perm"][b].long()] = torch.repeat_interleave(torch.arange(nb, device="cuda"), off[1:] - off[:-1])
        sel = torch.zeros(nb, nb, dtype=torch.bool, device="cuda")
        ptr = v["row_ptr"][(b * self.heads + h) * nbmax:][:nb + 1].tolist()
        for i in range(nb):
            sel[i, v["col_idx"][ptr[i]:ptr[i + 1]].long()] = True
        seen = sel[blk][:, blk]
        if self.doc is not None:
            seen &= (self.doc[b][:, None] == self.doc[b]) & (self.doc[b] >= 0)
        if self.causal:
            p = self.position[b]
            seen &= (p <= p[:, None]) | (p < (self.prefix[b] if self.prefix is not None else -math.inf))
        return seen

    def reference(self, b, h, q=None, k=None, v=None):
        """O, lse, (dQ, dK, dV) and the bounds of their errors, of head h of sample b."""
        q, k, v = (x[b, :, h].double() if y is None else y for x, y in ((self.Q, q), (self.K, k), (self.V, v)))
        do = self.dO[b, :, h].double()
        if self.doc is not None:  # what padding holds does not matter
            pad = (self.doc[b] < 0)[:, None]
            q, k, v, do = (x.masked_fill(pad, 0) for x in (q, k, v, do))
        scale = 1 / math.sqrt(self.dim)
        x = q @ k.T * scale
        d = torch.ones_like(x)
        if self.cap:
            t = torch.tanh(x / self.cap)
            x, d = self.cap * t, 1 - t * t
        if self.slopes is not None:
            p = self.position[b]
            x = x - float(self.slopes[h]) * (p[:, None] - p).abs()
        x = x.masked_fill(~self.allowed(b, h), -math.inf)
        lse = torch.logsumexp(x, 1)
        w = torch.exp(x - torch.where(lse.isfinite(), lse, 0)[:, None])
        O = w @ v
        eO = (E + FP32) * (w @ v.abs()) + E * O.abs()
        ds = w * (do @ v.T - (do * O).sum(1, keepdim=True)) * d
        eds = (E + FP32) * ds.abs() + w * d * ((do.abs() * eO).sum(1, keepdim=True) + FP32 * (do.abs() @ v.abs().T))
        dQ, dK, dV = ds @ k * scale, ds.T @ q * scale, w.T @ do
        eQ = scale * (eds @ k.abs()) + E * dQ.abs()
        eK = scale * (eds.T @ q.abs()) + E * dK.abs()
        eV = (E + FP32) * (w.T @ do.abs()) + E * dV.abs()
        return dict(O=O, lse=lse, dQ=dQ, dK=dK, dV=dV), dict(O=eO, dQ=eQ, dK=eK, dV=eV)

    def run(self, backward=True):
        O, lse = self.plan.fwd(scored=True)
        out = dict(O=O, lse=lse)
        if backward:
            out.update(zip(("dQ", "dK", "dV"), self.plan.bwd(O, self.dO, scored=True)))
        torch.cuda.synchronize()
        self.plan.check()
        return out

    def check(self, backward=True):
        got = self.run(backward)
        empty = 0
        for b in range(self.batch):
            for h in range(self.heads):
                ref, err = self.reference(b, h)
                lse = got["lse"][b, h].double()
                none = ref["lse"] == -math.inf
                empty += int(none.sum())
                assert torch.equal(lse == -math.inf, none)
                # fp32 logits: cap's tanh fit 4e-7 cap, products and bias a few 2^-24 of up to ~100
                assert ((lse - ref["lse"])[~none].abs() < 1e-4).all()
                for n in err if backward else ["O"]:
                    x = got[n][b, :, h].double()
                    off = (x - ref[n]).abs()
                    assert (off <= err[n] + 1e-30).all(), (n, b, h, (off - err[n]).max().item(), off.max().item())
                assert (got["O"][b, none][:, h] == 0).all()
                if backward:
                    assert (got["dQ"][b, none][:, h] == 0).all()
                    if self.doc is not None:
                        pad = self.doc[b] < 0
                        assert (got["dK"][b, pad][:, h] == 0).all() and (got["dV"][b, pad][:, h] == 0).all()
        return got, empty


FORMS = {
    "plain": dict(),
    "cap": dict(cap=8.0),
    "bias": dict(slope=0.7),
    "cap+bias": dict(cap=20.0, slope=0.3, pos="given"),
    "causal": dict(causal=True),
    "prefix": dict(causal=True, prefix=2),
    "clips": dict(clips=3),
    "clips+padding": dict(clips=2, padding=2),
    "tokens": dict(clips=4, padding=1, shuffled=True),
    "all": dict(cap=15.0, slope=0.4, clips=3, padding=1, causal=True, prefix=0.5, pos="given", shuffled=True),
    "all frames": dict(cap=50.0, slope=0.1, clips=2, padding=3, causal=True, prefix=1),
}
GRIDS = {
    "one zone": dict(T=8, H=8, W=8, heads=1, dim=64, frac=0.0),
    "tiny": dict(T=8, H=16, W=16, heads=2, dim=64),
    "odd": dict(T=16, H=8, W=24, heads=3, dim=128, top_k=2, frac=0.3),
    "batch": dict(T=8, H=16, W=8, heads=1, dim=128, batch=2),
    "hilbert": dict(T=16, H=16, W=8, heads=2, dim=64, hilbert=64, top_k=5),
}


@pytest.mark.gpu
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("grid", list(GRIDS))
def test_against_the_definition(P, grid, form):
    c = Case(P, **{**GRIDS[grid], **FORMS[form]}, seed=len(grid) * 31 + len(form))
    c.check()
    c.plan.close()


@pytest.mark.gpu
def test_rows_without_a_key(P):
    """Causal and clipped so hard that whole rows, whole tiles and whole blocks see nothing."""
    c = Case(P, 16, 16, 8, 2, 64, top_k=1, frac=0.01, causal=True, clips=5, padding=2, seed=3)
    _, empty = c.check()
    assert empty > 1000
    c.plan.update_qkv(c.Q, c.K, c.V)
    c.plan.set_score(doc=torch.full((1, c.N), -1, dtype=torch.int32, device="cuda"))  # nothing but padding
    c.doc, c.causal = torch.full((1, c.N), -1, dtype=torch.int32, device="cuda"), False
    _, empty = c.check()
    assert empty == 2 * c.N
    c.plan.close()


@pytest.mark.gpu
def test_what_padding_holds_reaches_nothing(P):
    c = Case(P, 16, 16, 8, 2, 128, clips=2, padding=4, causal=True, cap=10.0, slope=0.2, seed=4)
    clean = c.run()
    pad = c.doc[0] < 0
    for x, bad in ((c.Q, math.nan), (c.K, math.inf), (c.V, math.nan), (c.dO, -math.inf)):
        x[0, pad] = bad
    c.plan.update_qkv(c.Q, c.K, c.V)  # selection and scores stay
    O, lse = c.plan.fwd(scored=True)
    O2 = O.clone()
    O2[0, pad] = math.nan             # a caller's O need not hold zeros there
    dirty = dict(zip(("dQ", "dK", "dV"), c.plan.bwd(O2, c.dO, scored=True)), O=O, lse=lse)
    for n in ("O", "lse", "dK", "dV"):
        assert torch.equal(dirty[n], clean[n]), n
    # dQ's partial sums are added in the order they arrive
    assert (dirty["dQ"].float() - clean["dQ"].float()).abs().max() <= E * clean["dQ"].float().abs().max()
    c.plan.close()


@pytest.mark.gpu
def test_other_documents_for_the_same_tokens(P):
    """Tokens that were padding under one score are themselves again under the next: the zeros that a scored forward
    writes over padding must not outlive it, so new scores need the tensors brought in again."""
    c = Case(P, 16, 16, 8, 2, 64, clips=2, padding=6, seed=16)
    c.plan.set_score(doc=c.doc)          # twice without a forward between them: nothing is zeroed yet
    c.run()
    with pytest.raises(P.PrismError, match="zeroed padding"):
        c.plan.set_score(causal=True)
    c.run()                              # the refused call has changed nothing
    c.plan.update_qkv(c.Q, c.K, c.V)
    c.doc, c.causal = None, True
    c.plan.set_score(causal=True)
    c.check()
    c.plan.close()


@pytest.mark.gpu
def test_a_captured_forward_behind_an_eager_update(P):
    c = Case(P, 16, 16, 8, 2, 64, clips=2, padding=4, seed=17)
    want = c.run(backward=False)
    out = torch.empty_like(c.Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.plan.fwd(out, scored=True, want_lse=False)
    pad = c.doc[0] < 0
    for x in (c.Q, c.K, c.V):
        x[0, pad] = math.nan
    c.plan.update_qkv(c.Q, c.K, c.V)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want["O"])
    c.plan.close()


@pytest.mark.gpu
def test_large_logits_and_far_positions(P):
    for kw in (dict(gain=12.0, cap=0.01), dict(gain=12.0, cap=1e5), dict(gain=12.0, slope=40.0), dict(gain=40.0, cap=50.0)):
        c = Case(P, 16, 8, 16, 2, 64, seed=5, **kw)
        O, lse = c.plan.fwd(scored=True)
        for h in range(2):
            ref, err = c.reference(0, h)
            # logits of up to ~5000 are fp32: off by 2^-24 of that each, and P by as much
            slack = 2e-3
            assert ((O[0, :, h].double() - ref["O"]).abs() <= err["O"] + slack * 8).all(), kw
            assert (lse[0, h].double() - ref["lse"]).abs().max() < 2 * slack, kw
        c.plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [-70.0, 0.0, 70.0])
def test_rows_far_from_the_fixed_reference(P, shift):
    """Logits around +-70: sums of exponentials far outside fp32's middle range, with masks and gradients.  The shift is
    one that no row sees: K gets a component along a direction in which every query has the same extent."""
    c = Case(P, 16, 8, 16, 2, 64, clips=2, causal=True, seed=18)
    c.Q[..., 0] = 8.0
    c.K[..., 0] = shift          # adds 8 shift / sqrt(64) = shift to every logit
    c.plan.update_qkv(c.Q, c.K, c.V)
    c.check()
    # one tile's rows out of range beside others in range
    c.K[:, : c.N // 2, :, 0] = 0.0
    c.plan.update_qkv(c.Q, c.K, c.V)
    c.check()
    c.plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("shift,power", [(35.0, 90), (50.0, 60), (0.0, 110), (-18.0, -60), (-30.0, -60), (0.0, -60)])
def test_large_and_small_values(P, shift, power):
    """V of 2^power under logits around `shift`: their products pass fp32's largest (or fall below its least normal)
    number where the exponentials are taken as they are, O itself does not.  O is linear in V: the result over 2^power
    has the bounds of power = 0."""
    c = Case(P, 16, 8, 16, 2, 64, clips=2, causal=True, seed=21)
    c.Q[..., 0] = 8.0
    c.K[..., 0] = shift
    c.plan.update_qkv(c.Q, c.K, c.V * 2.0 ** power)  # a power of two: nothing is rounded
    O, _ = c.plan.fwd(scored=True)
    c.plan.check()
    for h in range(2):
        ref, err = c.reference(0, h)
        off = (O[0, :, h].double() * 2.0 ** -power - ref["O"]).abs()
        assert (off <= err["O"] + 1e-30).all(), (h, (off - err["O"]).max().item())
    c.plan.close()


@pytest.mark.gpu
def test_without_scores_it_is_the_sparse_attention(P):
    """No cap, bias or mask: fwd() and bwd() and their scored forms compute the same thing.  The two forwards round P
    against different reference maxima, so they may differ by the sum of their bounds, no more."""
    c = Case(P, 16, 16, 16, 2, 128, seed=6)
    scored, _ = c.check()
    O, lse = c.plan.fwd()
    dQ, dK, dV = c.plan.bwd(O, c.dO)
    for h in range(2):
        ref, err = c.reference(0, h)
        for n, x in (("O", O), ("dQ", dQ), ("dK", dK), ("dV", dV)):
            assert ((x[0, :, h].double() - ref[n]).abs() <= err[n] + 1e-30).all(), n
            assert ((x[0, :, h].double() - scored[n][0, :, h].double()).abs() <= 2 * err[n] + 1e-30).all(), n
    assert (lse - scored["lse"]).abs().max() < 2e-4
    c.plan.close()


@pytest.mark.gpu
def test_gradients_against_differences(P):
    """The 64-bit definition's gradients, which the kernel is held to above, against central differences of its output."""
    c = Case(P, 8, 8, 8, 1, 64, cap=6.0, slope=0.3, clips=2, causal=True, seed=7, frac=0.0)
    ref, _ = c.reference(0, 0)
    base = {n: x[0, :, 0].double() for n, x in (("q", c.Q), ("k", c.K), ("v", c.V))}
    do = c.dO[0, :, 0].double()
    h = 1e-5
    rs = np.random.default_rng(0)
    for name, grad in (("q", "dQ"), ("k", "dK"), ("v", "dV")):
        for _ in range(12):
            n, d = int(rs.integers(c.N)), int(rs.integers(64))
            vals = []
            for sign in (1, -1):
                x = base[name].clone()
                x[n, d] += sign * h
                vals.append((c.reference(0, 0, **{**base, name: x})[0]["O"] * do).sum())
            assert abs((vals[0] - vals[1]) / (2 * h) - ref[grad][n, d]) < 1e-6
    c.plan.close()


@pytest.mark.gpu
def test_graph_replay_and_another_stream(P):
    c = Case(P, 16, 16, 8, 2, 64, cap=10.0, clips=2, causal=True, slope=0.2, seed=8)
    want = c.run()
    outs = [torch.empty_like(c.Q) for _ in range(4)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.plan.update_qkv(c.Q, c.K, c.V)
        c.plan.set_score(cap=10.0, slopes=c.slopes, doc=c.doc, causal=True)
        c.plan.fwd(outs[0], scored=True, want_lse=False)
        c.plan.bwd(outs[0], c.dO, *outs[1:], scored=True)
    for x in outs:
        x.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want["O"]) and torch.equal(outs[2], want["dK"]) and torch.equal(outs[3], want["dV"])
    with torch.cuda.stream(s):
        O, _ = c.plan.fwd(scored=True)
    s.synchronize()
    assert torch.equal(O, want["O"])
    c.plan.close()


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused(P):
    """(One GPU: what the calls are given only says that it lies elsewhere, and is never read.)"""
    from types import SimpleNamespace

    from dynamic_block_sparse_zone_b200 import binding as B
    away = SimpleNamespace(device=torch.device("cuda", torch.cuda.current_device() + 1))
    B._here(doc=None, pos=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="slopes is on cuda"):
        B._here(doc=None, slopes=away)


@pytest.mark.gpu
def test_refusals(P):
    c = Case(P, 8, 16, 16, 2, 64, seed=9)
    plan = c.plan
    bad = [dict(cap=-1.0), dict(cap=float("nan")), dict(cap=1e-6), dict(prefix=torch.zeros(1, device="cuda"))]
    for kw in bad:
        with pytest.raises(P.PrismError, match="INVALID_ARG"):
            plan.set_score(**kw)
    for kw in (dict(slopes=torch.zeros(3, device="cuda")), dict(doc=torch.zeros(1, c.N, device="cuda")),
               dict(pos=torch.zeros(1, c.N)), dict(causal=True, prefix=torch.zeros(2, device="cuda"))):
        with pytest.raises(ValueError):
            plan.set_score(**kw)
    plan.set_score(cap=5.0)
    with pytest.raises(P.PrismError, match="ERR_STATE"):
        plan.bwd(c.Q, c.dO, scored=True)          # no scored forward yet
    O, _ = plan.fwd(scored=True)
    with pytest.raises(P.PrismError, match="ERR_STATE"):
        plan.bwd(O, c.dO)                         # the last forward was scored
    plan.fwd()
    with pytest.raises(P.PrismError, match="ERR_STATE"):
        plan.bwd(O, c.dO, scored=True)            # the last forward was not
    with pytest.raises(ValueError):
        plan.fwd(taylor=True, scored=True)
    plan.build(c.Q, c.K, c.V, torch.rand(1, 8, 16, 16, device="cuda"))
    with pytest.raises(P.PrismError, match="set_score"):
        plan.fwd(scored=True)                     # a build drops the scores
    fresh = P.PrismPlan(plan.params)
    with pytest.raises(P.PrismError, match="ERR_STATE"):
        fresh.set_score(cap=5.0)
    fresh.build(c.Q, c.K, c.V, torch.rand(1, 8, 16, 16, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(P.PrismError, match="capture"):
            fresh.set_score(cap=5.0)              # its first call allocates
        fresh.fwd(want_lse=False)
    fresh.set_score(cap=5.0)
    fresh.fwd(scored=True)
    torch.cuda.synchronize()
    plan.close()
    fresh.close()


def test_null_arguments_are_rejected(P):
    lib = P.load_library()
    assert lib.prism_plan_set_score(None, None, None) == 1
    assert lib.prism_attn_fwd_scored(None, None, None, None) == 1
    assert lib.prism_attn_bwd_scored(None, None, None, None, None, None, None) == 1
    assert b"NULL" in lib.prism_last_error()
