"""Attention checkpoints in 8 bits: what they hold, and the backward that reads them, against the
definition in 64 bits (bounds as in test_scored_gpu.py; O is given exactly, so Delta adds only fp32)."""
import math

import numpy as np
import pytest
import torch

from test_scored_gpu import E, FP32, Case

FORMS = {
    "sparse": None,
    "scored": dict(cap=12.0, slope=0.3, clips=2, causal=True, prefix=1),
    "padded": dict(clips=3, padding=2),
}
GRIDS = {
    "tiny": dict(T=8, H=16, W=16, heads=2, dim=64),
    "odd": dict(T=16, H=8, W=24, heads=3, dim=128, top_k=2, frac=0.3),
    "batch": dict(T=8, H=16, W=8, heads=1, dim=128, batch=2),
    "hilbert": dict(T=16, H=16, W=8, heads=2, dim=64, hilbert=128),
}


@pytest.fixture(scope="module")
def P():
    from dynamic_block_sparse_zone_b200 import build as b
    b.build()
    import dynamic_block_sparse_zone_b200 as P
    P.load_library()
    return P


def definition(c, b, h, vals, lse, scored):
    """dQ, dK, dV from 8-bit values (q, k, v, o) and the saved lse, and bounds of the kernel's errors."""
    q, k, v, o = (x[b, :, h].double() for x in vals)
    do = c.dO[b, :, h].double()
    if scored and c.doc is not None:
        pad = (c.doc[b] < 0)[:, None]
        q, k, v, o, do = (x.masked_fill(pad, 0) for x in (q, k, v, o, do))
    scale = 1 / math.sqrt(c.dim)
    x = q @ k.T * scale
    d = torch.ones_like(x)
    if scored and c.cap:
        t = torch.tanh(x / c.cap)
        x, d = c.cap * t, 1 - t * t
    if scored and c.slopes is not None:
        p = c.position[b]
        x = x - float(c.slopes[h]) * (p[:, None] - p).abs()
    keep = c.doc, c.causal
    if not scored:
        c.doc, c.causal = None, False
    seen = c.allowed(b, h)
    c.doc, c.causal = keep
    l = lse[b, h].double()
    w = torch.exp(x - torch.where(l.isfinite(), l, 0)[:, None]).masked_fill(~seen, 0)
    ds = w * (do @ v.T - (do * o).sum(1, keepdim=True)) * d
    eds = (E + FP32) * ds.abs() + FP32 * w * d * ((do * o).abs().sum(1, keepdim=True) + do.abs() @ v.abs().T)
    dQ, dK, dV = ds @ k * scale, ds.T @ q * scale, w.T @ do
    return ((dQ, scale * (eds @ k.abs()) + E * dQ.abs()), (dK, scale * (eds.T @ q.abs()) + E * dK.abs()),
            (dV, (E + FP32) * (w.T @ do.abs()) + E * dV.abs()))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("grid", list(GRIDS))
def test_backward_from_a_checkpoint(P, grid, form, fmt):
    scored = FORMS[form] is not None
    c = Case(P, **{**GRIDS[grid], **(FORMS[form] or {})}, seed=len(grid) + 7 * len(form))
    if scored and c.doc is not None:  # padding may hold anything
        pad = c.doc < 0
        for x in (c.Q, c.K, c.V):
            x[pad] = math.nan
        c.dO[pad] = math.inf
        c.plan.update_qkv(c.Q, c.K, c.V)
    O, lse = c.plan.fwd(scored=scored)
    kept = c.plan.save(c.Q, c.K, c.V, O, lse, fmt)
    assert kept.nbytes - lse.nbytes == 4 * c.Q.numel() * 33 // 32
    for part, x in zip((kept.Q, kept.K, kept.V, kept.O), (c.Q, c.K, c.V, O)):
        one = P.prism_ckpt_pack(x.reshape(-1, c.heads * c.dim), fmt)
        assert torch.equal(part.codes, one.codes) and torch.equal(part.scales, one.scales)
    vals = [P.prism_ckpt_unpack(k) for k in (kept.Q, kept.K, kept.V, kept.O)]
    # something else passes through the plan before the backward
    other = torch.randn(c.Q.shape, device="cuda").bfloat16()
    c.plan.update_qkv(other, other, other)
    c.plan.fwd(scored=scored)
    got = c.plan.bwd_ckpt(kept, c.dO, scored=scored)
    torch.cuda.synchronize()
    c.plan.check()
    for b in range(c.batch):
        for h in range(c.heads):
            for n, g, (want, bound) in zip(("dQ", "dK", "dV"), got, definition(c, b, h, vals, lse, scored)):
                off = (g[b, :, h].double() - want).abs()
                assert (off <= bound + 1e-30).all(), (n, b, h, (off - bound).max().item(), off.max().item())
    # the exact gradient at the 8-bit point, and the forward there
    c.plan.update_qkv_ckpt(kept)
    O1, lse1 = c.plan.fwd(scored=scored)
    g1 = c.plan.bwd(O1, c.dO, scored=scored)
    c.plan.update_qkv(*vals[:3])
    O2, lse2 = c.plan.fwd(scored=scored)
    g2 = c.plan.bwd(O2, c.dO, scored=scored)
    assert torch.equal(O1, O2) and torch.equal(lse1, lse2) and torch.equal(g1[1], g2[1]) and torch.equal(g1[2], g2[2])
    c.plan.close()


@pytest.mark.gpu
def test_the_taylor_forward_after_a_checkpoint(P):
    """update_qkv_ckpt refreshes the pooled keys as update_qkv does."""
    c = Case(P, 16, 16, 16, 2, 64, frac=0.25, seed=11)
    O, lse = c.plan.fwd()
    kept = c.plan.save(c.Q, c.K, c.V, O, lse, "e4m3")
    vals = [P.prism_ckpt_unpack(k) for k in (kept.Q, kept.K, kept.V)]
    c.plan.update_qkv_ckpt(kept)
    a = c.plan.fwd(taylor=True)
    c.plan.update_qkv(*vals)
    b = c.plan.fwd(taylor=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.plan.close()


@pytest.mark.gpu
def test_how_far_the_gradient_moves(P):
    """Against the gradient without checkpoints: an int8 value is off by at most 2^(k-1) with max|x| > 63.5 * 2^k of its
    group, that is max|x| / 127; with N(0, s) inputs (max|x| of 32 about 2.1 s) uniform errors have a standard deviation of
    at most 2.1 s / 127 / sqrt(3) = 0.0096 s.  Logits (s = 1.2: standard deviation 1.44, 64 products) then move by
    0.0096 * sqrt(2) * 1.44 = 0.020, and P, dP and Delta by about 2% each: 5% of the gradients' norm is over twice that."""
    c = Case(P, 16, 16, 16, 2, 64, gain=1.2, seed=12)
    O, lse = c.plan.fwd()
    want = c.plan.bwd(O, c.dO)
    got = c.plan.bwd_ckpt(c.plan.save(c.Q, c.K, c.V, O, lse, "int8"), c.dO)
    for g, w in zip(got, want):
        assert (g.float() - w.float()).norm() <= 0.05 * w.float().norm()
    c.plan.close()


@pytest.mark.gpu
def test_a_layers_training_step(P):
    """The operators together, as a layer uses them: norm of the stream, projections, per-head norms, scored attention
    on packed clips, everything kept in 8 bits, and back; against the same step in 64 bits on the 8-bit values."""
    T, H, W, heads, dim = 8, 16, 16, 2, 64
    N, C = T * H * W, heads * dim
    g = torch.Generator(device="cuda").manual_seed(13)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (rand(1, N, C) * 2 + 0.3).bfloat16()
    w = (rand(C, 3 * C) / math.sqrt(C)).bfloat16()
    gamma, beta = 1 + 0.1 * rand(C), 0.1 * rand(C)
    qg = 1 + 0.1 * rand(dim)
    dO = rand(1, N, heads, dim).bfloat16()
    y, mean, rstd, xk = P.prism_layer_norm_fwd(x, gamma, beta, ckpt="int8")
    qkv = (y @ w).view(1, N, 3, heads, dim)
    q, qm, qr, qk = P.prism_layer_norm_fwd(qkv[:, :, 0], qg, ckpt="int8")    # heads of a fused projection
    k, km, kr, kk = P.prism_layer_norm_fwd(qkv[:, :, 1], qg, ckpt="int8")
    v = qkv[:, :, 2].contiguous()
    plan = P.PrismPlan(P.Params(batch=1, T=T, H=H, W=W, heads=heads, head_dim=dim, top_k=4, top_p=0.9, max_frac=0.5))
    plan.build(q, k, v, rand(1, T, H, W).abs())
    doc = (torch.arange(N, device="cuda") // (3 * H * W)).int()[None]
    plan.set_score(cap=10.0, slopes=torch.full((heads,), 0.1, device="cuda"), doc=doc, causal=True)
    O, lse = plan.fwd(scored=True)
    kept = plan.save(q, k, v, O, lse)
    dq, dk, dv = plan.bwd_ckpt(kept, dO, scored=True)
    dqkv = torch.zeros_like(qkv)
    dq0, dqg, _ = P.prism_layer_norm_bwd(dq, qk, qg, qm, qr, dx=dqkv[:, :, 0])
    dk0, dkg, _ = P.prism_layer_norm_bwd(dk, kk, qg, km, kr, dx=dqkv[:, :, 1])
    dqkv[:, :, 2] = dv
    dy = (dqkv.view(1, N, 3 * C) @ w.T)
    dx, dgamma, dbeta = P.prism_layer_norm_bwd(dy, xk, gamma, mean, rstd)

    # the same step in 64 bits, autograd through the whole of it, without any rounding or 8 bits
    X = x.double().requires_grad_()
    G, B, QG = (t.double().requires_grad_() for t in (gamma, beta, qg))
    norm = lambda t, a, b: torch.nn.functional.layer_norm(t, t.shape[-1:], a, b, 1e-6)  # noqa: E731
    QKV = (norm(X, G, B) @ w.double()).view(N, 3, heads, dim)
    Q, K, V = norm(QKV[:, 0], QG, None), norm(QKV[:, 1], QG, None), QKV[:, 2]
    c = Case.__new__(Case)
    c.plan, c.N, c.heads, c.doc, c.causal, c.prefix = plan, N, heads, doc, True, None
    frame = torch.arange(N, device="cuda") // (H * W)
    c.position = frame.double()[None]
    loss = 0.0
    for h in range(heads):
        s = 10 * torch.tanh(Q[:, h] @ K[:, h].T / math.sqrt(dim) / 10) - 0.1 * (frame[:, None] - frame).abs()
        s = s.masked_fill(~c.allowed(0, h), -math.inf)
        loss = loss + (torch.softmax(s, 1).nan_to_num(0) @ V[:, h] * dO[0, :, h].double()).sum()
    want = torch.autograd.grad(loss, (X, G, B, QG))
    # bf16 activations (2^-8 each through seven roundings in a row: under 3%) and int8 (each value off by under 1% of its
    # group's largest, as in the test above: about 2% in P, dP, Delta and the norms' inputs): 8% bounds their sum
    for n, a, b in (("x", dx, want[0]), ("gamma", dgamma, want[1]), ("beta", dbeta, want[2]), ("qk gamma", dqg + dkg, want[3])):
        assert (a.double() - b).norm() <= 0.08 * b.norm(), (n, ((a.double() - b).norm() / b.norm()).item())
    plan.close()


@pytest.mark.gpu
def test_graph_of_the_step(P):
    c = Case(P, 8, 16, 16, 2, 64, seed=14, cap=9.0, causal=True)
    O, lse = c.plan.fwd(scored=True)
    kept = c.plan.save(c.Q, c.K, c.V, O, lse)
    want = c.plan.bwd_ckpt(kept, c.dO, scored=True)
    outs = [torch.full_like(c.Q, 7) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.plan.update_qkv(c.Q, c.K, c.V)
        O2, lse2 = c.plan.fwd(scored=True)
        k2 = c.plan.save(c.Q, c.K, c.V, O2, lse2)
        c.plan.bwd_ckpt(k2, c.dO, *outs, scored=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], want[1]) and torch.equal(outs[2], want[2])
    c.plan.close()


@pytest.mark.gpu
def test_refusals(P):
    c = Case(P, 8, 16, 16, 2, 64, seed=15)
    O, lse = c.plan.fwd()
    kept = c.plan.save(c.Q, c.K, c.V, O, lse)
    with pytest.raises(ValueError):
        c.plan.save(c.Q, c.K, c.V, O, lse, "int4")
    with pytest.raises(ValueError):
        c.plan.save(c.Q.float(), c.K, c.V, O, lse)
    with pytest.raises(ValueError):
        c.plan.bwd_ckpt(kept, c.dO[:, :64])
    small = P.PrismPlan(P.Params(batch=1, T=8, H=8, W=8, heads=2, head_dim=64, top_k=1, top_p=0.9))
    with pytest.raises(ValueError, match="other sizes"):
        small.bwd_ckpt(kept, c.dO[:, :512])
    fresh = P.PrismPlan(c.plan.params)
    for call in (lambda: fresh.update_qkv_ckpt(kept), lambda: fresh.bwd_ckpt(kept, c.dO)):
        with pytest.raises(P.PrismError, match="ERR_STATE"):
            call()
    c.plan.build_with_zones(c.Q, c.K, c.V, np.full((1, 4), 64), np.full((1, 4), 0))
    with pytest.raises(P.PrismError, match="set_score"):
        c.plan.bwd_ckpt(kept, c.dO, scored=True)  # the build dropped the scores
    c.plan.bwd_ckpt(kept, c.dO)
    with pytest.raises(P.PrismError, match="ERR_STATE"):
        c.plan.bwd(O, c.dO)                       # the plan holds the checkpoint's Q, K, V now
    torch.cuda.synchronize()


def test_arguments_are_checked_on_the_host(P):
    from dynamic_block_sparse_zone_b200 import binding as B
    import ctypes
    lib = P.load_library()
    c = ctypes.byref(B.prism_attn_ckpt())
    assert lib.prism_attn_ckpt_save(None, None, None, None, None, c, None) == 1
    assert lib.prism_plan_update_qkv_ckpt(None, c, None) == 1
    assert lib.prism_attn_bwd_ckpt(None, c, None, None, None, None, 0, None) == 1
    assert b"NULL" in lib.prism_last_error()
