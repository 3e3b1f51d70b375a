"""Timed cases of the operators around one video attention layer in training:

* layer norm of the token stream and of the heads, forward and backward;
* 8-bit checkpoints of activations, and the backward passes that read them;
* block-sparse attention whose scores are capped, biased by distance, and masked by
  packed clips, padding, causality and a prefix, forward and backward.

Every case runs in two forms on the same inputs: the plain one (elementary torch
operations in 32 bits, rounded once at the end) and, with ``own`` set, the library's.
``exact`` is the operators' definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GROUP = 32                                    # channels that share one scale of a checkpoint
QMAX = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
TOP_P = 0.9375
# the block shapes (frames, rows, columns) of 64, 128 and 256 tokens with edges 2, 4 and 8
SHAPES = [(a, b, c) for v in (64, 128, 256) for a in (2, 4, 8) for b in (2, 4, 8) for c in (2, 4, 8) if a * b * c == v]


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a single token's hidden state, as a step that appends one token norms it: latency
        dict(name="norm_fwd_one_token", op="norm", way="fwd", rows=1, channels=1024, dtype="bf16", weights="bf16", pad=0),
        # query/key norm of every head of a 16x32x32 latent's tokens (8 heads of 128)
        dict(name="norm_fwd_heads", op="norm", way="fwd", rows=131072, channels=128, dtype="bf16", weights="fp32", pad=0),
        # the hidden stream of a 720p-like latent (24x48x80 tokens)
        dict(name="norm_fwd_latent", op="norm", way="fwd", rows=92160, channels=1536, dtype="bf16", weights="fp32", pad=0),
        # a ragged batch in fp32 whose rows are a slice of wider ones
        dict(name="norm_bwd_ragged", op="norm", way="bwd", rows=4099, channels=1000, dtype="fp32", weights="fp32", pad=24),
        # the gradient of the hidden stream's norm at the same latent
        dict(name="norm_bwd_latent", op="norm", way="bwd", rows=92160, channels=2048, dtype="bf16", weights="fp32", pad=0),
        # a training step of that norm whose input is kept in 8 bits between the passes
        dict(name="norm_step_checkpoint", op="norm", way="step", rows=65536, channels=2048, dtype="bf16", weights="bf16", pad=0, fmt="int8"),
        # one frame's activations written to 8 bits and read back: latency
        dict(name="checkpoint_frame", op="pack", rows=1024, channels=1000, dtype="fp16", pad=0, fmt="int8"),
        # a whole latent's activations written to 8 bits and read back
        dict(name="checkpoint_latent", op="pack", rows=92160, channels=2048, dtype="bf16", pad=0, fmt="e4m3"),
        # an attention layer's training step that keeps Q, K, V and O in 8 bits in between
        dict(name="attention_step_checkpoint", op="attn", way="checkpoint", T=16, H=32, W=32, heads=8, dim=128, top_k=8, frac=0.25,
             fmt="int8", cap=0.0, slope=0.0, clips=0, padding=0, causal=False, prefix=0),
        # a tiny latent sampled frame by frame: causal after a two-frame prefix
        dict(name="attention_fwd_causal", op="attn", way="fwd", T=8, H=16, W=16, heads=2, dim=64, top_k=4, frac=0.5,
             fmt="", cap=0.0, slope=0.0, clips=0, padding=0, causal=True, prefix=2),
        # capped scores that fall with the distance in frames, no mask
        dict(name="attention_fwd_capped", op="attn", way="fwd", T=16, H=32, W=32, heads=8, dim=128, top_k=8, frac=0.25,
             fmt="", cap=20.0, slope=0.25, clips=0, padding=0, causal=False, prefix=0),
        # a training step on three clips packed along time with padded frames behind them, everything on
        dict(name="attention_step_packed", op="attn", way="step", T=24, H=32, W=40, heads=2, dim=128, top_k=16, frac=0.25,
             fmt="", cap=30.0, slope=0.125, clips=3, padding=1, causal=True, prefix=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pack", "attn", "attn"])
    if op in ("norm", "pack"):
        channels = rng.choice([64, 128, _log(rng, 8, 8192), 8 * _log(rng, 8, 640)])
        rows = _log(rng, 1, max(1, min(131072, (92160 * 2048) // (2 * channels))))
        case = dict(op=op, rows=rows, channels=channels, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    pad=rng.choice([0, 0, 0, 8, rng.randrange(1, 40)]), fmt=rng.choice(["int8", "e4m3"]))
        if op == "norm":
            case["way"] = rng.choice(["fwd", "bwd", "step"])
            case["weights"] = rng.choice(["fp32", case["dtype"]])
        return case
    way = rng.choice(["fwd", "step", "checkpoint"])
    heads, dim = rng.randrange(1, 7), rng.choice([64, 128])
    while True:
        T, H, W = 8 * rng.randrange(1, 4), 8 * rng.randrange(1, 6), 8 * rng.randrange(1, 6)
        if heads * (T * H * W) ** 2 <= 1.6e9:
            break
    return dict(op="attn", way=way, T=T, H=H, W=W, heads=heads, dim=dim, top_k=rng.randrange(1, 17),
                frac=rng.choice([0.125, 0.25, 0.5]), fmt=rng.choice(["int8", "e4m3"]),
                cap=rng.choice([0.0, rng.uniform(5.0, 50.0)]), slope=rng.choice([0.0, rng.uniform(0.02, 1.0)]),
                clips=rng.choice([0, 1, 2, 3]), padding=rng.choice([0, 0, 1, 3]), causal=rng.random() < 0.5,
                prefix=rng.choice([0, 1, 3]))


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rows(case, g, scale, offset):
    """rows x channels activations: per-channel scales spread over a decade, a few loud channels,
    an offset per row; stored inside rows that are `pad` channels wider."""
    r, c = case["rows"], case["channels"]
    x = torch.randn(r, c, generator=g, device=DEV)
    gain = torch.exp(torch.randn(c, generator=g, device=DEV) * 0.5) * scale
    gain[torch.rand(c, generator=g, device=DEV) < 0.01] *= 8
    x = x * gain + offset * torch.randn(r, 1, generator=g, device=DEV) + offset
    wide = torch.zeros(r, c + case["pad"], dtype=DTYPE[case["dtype"]], device=DEV)
    wide[:, :c] = x
    return wide[:, :c]


def _norm_inputs(case, seed):
    g = _gen(seed)
    c = case["channels"]
    s = dict(x=_rows(case, g, 1.0, 0.5))
    s["gamma"] = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).to(DTYPE[case["weights"]])
    s["beta"] = (0.2 * torch.randn(c, generator=g, device=DEV)).to(DTYPE[case["weights"]])
    if case["way"] != "fwd":
        s["dy"] = _rows(case, g, 0.1, 0.01)
    if case["way"] == "bwd":  # the statistics that the forward pass has kept
        x = s["x"].double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = ((x - x.mean(1, keepdim=True)).square().mean(1) + EPS).rsqrt().float()
    return s


def _smooth(case, g, channels):
    """[N, channels] field over the grid: two slow waves per channel and noise."""
    T, H, W = case["T"], case["H"], case["W"]
    t, h, w = (torch.arange(n, device=DEV, dtype=torch.float32) / n for n in (T, H, W))
    out = torch.randn(T, H, W, channels, generator=g, device=DEV) * 0.6
    f = torch.rand(2, 3, channels, generator=g, device=DEV) * 3 * 2 * math.pi
    ph = torch.rand(2, channels, generator=g, device=DEV) * 2 * math.pi
    at = t[:, None, None, None, None] * f[:, 0] + h[:, None, None, None] * f[:, 1] + w[:, None, None] * f[:, 2] + ph
    return (out + at.sin().sum(3)).reshape(T * H * W, channels)


def _attn_inputs(case, seed):
    g = _gen(seed)
    N, heads, dim = case["T"] * case["H"] * case["W"], case["heads"], case["dim"]
    s = dict(case=case)
    for name, gain in (("Q", 1.5), ("K", 1.5), ("V", 1.0)):
        s[name] = (gain * _smooth(case, g, heads * dim)).reshape(1, N, heads, dim).bfloat16()
    if case["way"] != "fwd":
        s["dO"] = torch.randn(1, N, heads, dim, generator=g, device=DEV).bfloat16()
    rs = np.random.default_rng(int(seed))
    # each 8x8x8 zone's block shape: given, as when one layer's decisions serve several
    s["shape"] = rs.integers(0, len(SHAPES), N // 512).astype(np.int32)
    s["volume"] = np.array([np.prod(SHAPES[i]) for i in s["shape"]], dtype=np.int32)
    # clips packed along time, each with its own frame count from zero, and padded frames last
    T, used = case["T"], max(1, case["T"] - case["padding"])
    cuts = sorted(rs.choice(np.arange(1, used), min(max(case["clips"], 1), used) - 1, replace=False)) if used > 1 else []
    doc = np.full(T, -1, dtype=np.int32)
    pos = np.zeros(T, dtype=np.float32)
    for i, (a, b) in enumerate(zip([0, *cuts], [*cuts, used])):
        doc[a:b], pos[a:b] = i, np.arange(b - a)
    rep = case["H"] * case["W"]
    s["doc"] = torch.from_numpy(np.repeat(doc, rep)[None]).to(DEV) if case["clips"] or case["padding"] else None
    s["pos"] = torch.from_numpy(np.repeat(pos, rep)[None]).to(DEV)
    s["slopes"] = (case["slope"] * 0.5 ** torch.arange(heads, device=DEV, dtype=torch.float32)) if case["slope"] else None
    s["prefix"] = torch.full((1,), float(case["prefix"]), device=DEV) if case["causal"] and case["prefix"] else None
    return s


def _scored(case):
    return bool(case["cap"] or case["slope"] or case["clips"] or case["padding"] or case["causal"])


def prepare(case, seed):
    if case["op"] == "norm":
        return dict(case=case, **_norm_inputs(case, seed))
    if case["op"] == "pack":
        return dict(case=case, x=_rows(case, _gen(seed), 1.0, 0.5))
    s = _attn_inputs(case, seed)
    if own:  # the plan that a program builds once for its layers, with its masks
        import dynamic_block_sparse_zone_b200 as P

        s["plan"] = P.PrismPlan(P.Params(batch=1, T=case["T"], H=case["H"], W=case["W"], heads=case["heads"], head_dim=case["dim"],
                                         top_k=case["top_k"], top_p=TOP_P, max_frac=case["frac"]))
        s["plan"].build_with_zones(s["Q"], s["K"], s["V"], s["volume"], s["shape"])
        if _scored(case) or case["way"] == "checkpoint":
            s["plan"].set_score(cap=case["cap"], slopes=s["slopes"], pos=s["pos"], doc=s["doc"], causal=case["causal"], prefix=s["prefix"])
    else:
        s["allowed"] = _plain_allowed(s)
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_8bit(x, fmt):
    """The values that x's 8-bit form stands for, in 32 bits: groups of 32 channels share the
    smallest power of two that brings their largest magnitude within the format's."""
    c = x.shape[-1]
    g = torch.nn.functional.pad(x.float(), (0, -c % GROUP)).unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)
    k = (e - 7 + (m > 127 / 128).int()) if fmt == "int8" else (e - 9 + (m > 448 / 512).int())
    k = torch.where(top.isfinite() & (top > 0), k, 0).clamp(min=-127).int()
    up, down = (k + 127).clamp(min=1) << 23, (127 - k) << 23  # the exponent bits of 2^k and 2^-k
    up, down = up.view(torch.float32) * torch.where(k == -127, 0.5, 1.0), down.view(torch.float32)
    y = g * down
    y = torch.round(y) if fmt == "int8" else y.to(torch.float8_e4m3fn).float()
    y = torch.where(top.isfinite(), y * up, math.nan)
    return y.flatten(-2)[..., :c]


def _plain_norm_fwd(x, gamma, beta):
    x = x.float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + EPS).rsqrt()
    return d * rstd[:, None] * gamma.float() + beta.float(), mean, rstd


def _plain_norm_bwd(x, dy, gamma, mean, rstd):
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    dy = dy.float()
    g = dy * gamma.float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd[:, None]
    return dx, (dy * xh).sum(0), dy.sum(0)


def _plain_allowed(s):
    """[heads, N, N] truth values: which keys each query attends to, from the block selection
    (pooled scores, the best k blocks or the most likely part TOP_P of the mass, at most a share of the blocks) and the masks."""
    case = s["case"]
    T, H, W, heads, dim = (case[k] for k in ("T", "H", "W", "heads", "dim"))
    N = T * H * W
    n = torch.arange(N, device=DEV)
    t, h, w = n // (H * W), n // W % H, n % W
    zone = ((t // 8) * (H // 8) + h // 8) * (W // 8) + w // 8
    edge = torch.tensor(SHAPES, device=DEV)[torch.from_numpy(s["shape"]).to(DEV).long()][zone]
    per = 512 // torch.from_numpy(s["volume"]).to(DEV).long()
    first = torch.cumsum(per, 0) - per
    blk = first[zone] + ((t % 8) // edge[:, 0] * (8 // edge[:, 1]) + (h % 8) // edge[:, 1]) * (8 // edge[:, 2]) + (w % 8) // edge[:, 2]
    nb = int(per.sum())
    size = torch.bincount(blk, minlength=nb).double()
    mean = [torch.zeros(nb, heads * dim, device=DEV, dtype=torch.float64).index_add_(0, blk, s[x][0].flatten(1).double()) / size[:, None] for x in ("Q", "K")]
    qb, kb = (m.unflatten(1, (heads, dim)).transpose(0, 1) for m in mean)
    z = qb @ kb.mT / math.sqrt(dim)
    best, order = z.sort(dim=2, descending=True, stable=True)
    mass = best.softmax(2).cumsum(2)
    keep = ((mass < TOP_P).sum(2) + 1).clamp(min=case["top_k"], max=max(case["top_k"], int(case["frac"] * nb))).clamp(max=nb)
    sel = torch.zeros(heads, nb, nb, dtype=torch.bool, device=DEV)
    sel.scatter_(2, order, torch.arange(nb, device=DEV) < keep[:, :, None])
    allowed = sel[:, blk][:, :, blk]
    if _scored(case):
        pos = s["pos"][0]
        if s["doc"] is not None:
            d = s["doc"][0]
            allowed &= (d[:, None] == d) & (d >= 0)
        if case["causal"]:
            allowed &= (pos <= pos[:, None]) | (pos < case["prefix"])
    return allowed


def _plain_attn(s, Q, K, V):
    """Scores' tanh (None without a cap), probabilities, output and log-sum-exp, [heads, ...]."""
    case = s["case"]
    x = (Q @ K.mT).mul_(1 / math.sqrt(case["dim"]))
    t = None
    if case["cap"]:
        t = (x / case["cap"]).tanh_()
        x = t * case["cap"]
    if s["slopes"] is not None:
        pos = s["pos"][0]
        x = x.sub_(s["slopes"][:, None, None] * (pos[:, None] - pos).abs())
    x = x.masked_fill_(~s["allowed"], -math.inf)
    m = x.amax(2, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = x.sub_(m).exp_()
    l = p.sum(2, keepdim=True)
    lse = (m + l.log())[..., 0]
    p = p.div_(torch.where(l == 0, 1, l))
    return t, p, p @ V, lse


def _plain_attn_grads(s, Q, K, V, t, p, dO, delta):
    dV = p.mT @ dO
    ds = (dO @ V.mT).sub_(delta).mul_(p)
    if t is not None:
        ds = ds.mul_(1 - t * t)
    ds = ds.mul_(1 / math.sqrt(s["case"]["dim"]))
    return ds @ K, ds.mT @ Q, dV


def _heads(x):
    return x[0].float().transpose(0, 1)


def _tokens(x):
    return x.transpose(0, 1)[None].bfloat16()


def _plain_attn_pass(s):
    way = s["case"]["way"]
    Q, K, V = (_heads(s[k]) for k in "QKV")
    t, p, O, lse = _plain_attn(s, Q, K, V)
    out = dict(O=_tokens(O), lse=lse[None])
    if way == "fwd":
        return out
    dO = _heads(s["dO"])
    if way == "checkpoint":  # the backward pass sees Q, K, V and O as their 8 bits stand for them
        fmt = s["case"]["fmt"]
        Q, K, V = (_plain_8bit(x, fmt) for x in (Q, K, V))
        O = _plain_8bit(O.bfloat16(), fmt)
        del p
        x = (Q @ K.mT).mul_(1 / math.sqrt(s["case"]["dim"]))
        if s["case"]["cap"]:
            t = (x / s["case"]["cap"]).tanh_()
            x = t * s["case"]["cap"]
        if s["slopes"] is not None:
            pos = s["pos"][0]
            x = x.sub_(s["slopes"][:, None, None] * (pos[:, None] - pos).abs())
        p = x.sub_(lse[:, :, None]).exp_().masked_fill_(~s["allowed"], 0)
    dQ, dK, dV = _plain_attn_grads(s, Q, K, V, t, p, dO, (dO * O).sum(2, keepdim=True))
    return dict(out, dQ=_tokens(dQ), dK=_tokens(dK), dV=_tokens(dV))


def _plain_run(s):
    case = s["case"]
    if case["op"] == "attn":
        return _plain_attn_pass(s)
    dt = DTYPE[case["dtype"]]
    if case["op"] == "pack":
        return _plain_8bit(s["x"], case["fmt"]).to(dt)
    out = {}
    if case["way"] != "bwd":
        y, mean, rstd = _plain_norm_fwd(s["x"], s["gamma"], s["beta"])
        out = dict(y=y.to(dt), mean=mean, rstd=rstd)
    if case["way"] != "fwd":
        x = s["x"]
        if case["way"] == "bwd":
            mean, rstd = s["mean"], s["rstd"]
        else:
            x = _plain_8bit(x, case["fmt"])
        dx, dgamma, dbeta = _plain_norm_bwd(x, s["dy"], s["gamma"], mean, rstd)
        out |= dict(dx=dx.to(dt), dgamma=dgamma.to(s["gamma"].dtype), dbeta=dbeta.to(s["gamma"].dtype))
    return out


# --------------------------------------------------------------------------- the library's calls
def _own_run(s):
    import dynamic_block_sparse_zone_b200 as P

    case = s["case"]
    if case["op"] == "pack":
        return P.prism_ckpt_unpack(P.prism_ckpt_pack(s["x"], case["fmt"]))
    if case["op"] == "norm":
        if case["way"] == "fwd":
            y, mean, rstd = P.prism_layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS)
            return dict(y=y, mean=mean, rstd=rstd)
        if case["way"] == "bwd":
            dx, dgamma, dbeta = P.prism_layer_norm_bwd(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])
            return dict(dx=dx, dgamma=dgamma, dbeta=dbeta)
        y, mean, rstd, kept = P.prism_layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, ckpt=case["fmt"])
        dx, dgamma, dbeta = P.prism_layer_norm_bwd(s["dy"], kept, s["gamma"], mean, rstd)
        return dict(y=y, mean=mean, rstd=rstd, dx=dx, dgamma=dgamma, dbeta=dbeta)
    plan, scored = s["plan"], _scored(case)
    plan.update_qkv(s["Q"], s["K"], s["V"])
    # an O that is kept in 8 bits comes from the scored forward, with or without scores: it is right to its last bit
    # (the sparse forward rounds its probabilities, and every tenth 8-bit code falls on the other side)
    O, lse = plan.fwd(scored=scored or case["way"] == "checkpoint")
    if case["way"] == "fwd":
        return dict(O=O, lse=lse)
    if case["way"] == "step":
        dQ, dK, dV = plan.bwd(O, s["dO"], scored=scored)
    else:
        kept = plan.save(s["Q"], s["K"], s["V"], O, lse, case["fmt"])
        dQ, dK, dV = plan.bwd_ckpt(kept, s["dO"], scored=scored)
    return dict(O=O, lse=lse, dQ=dQ, dK=dK, dV=dV)


def run(state):
    return _own_run(state) if own else _plain_run(state)


# --------------------------------------------------------------------------- work
def work(case):
    if case["op"] != "attn":
        n, es = case["rows"] * case["channels"], SIZE[case["dtype"]]
        kept = 1 + 1 / GROUP
        if case["op"] == "pack":
            return {"bytes": n * (2 * es + 2 * kept), "flops": 4 * n}
        small = 2 * case["channels"] * SIZE[case["weights"]] + 8 * case["rows"]
        if case["way"] == "fwd":
            return {"bytes": n * 2 * es + small, "flops": 8 * n}
        if case["way"] == "bwd":
            return {"bytes": n * 3 * es + 1.5 * small, "flops": 14 * n}
        return {"bytes": n * (4 * es + 2 * kept) + 2.5 * small, "flops": 26 * n}
    N = case["T"] * case["H"] * case["W"]
    # pairs of the selection's cap, and of them those that the masks leave if the selection is blind to the masks
    pairs = case["heads"] * N * N * min(1.0, max(case["frac"], case["top_k"] * 110 / N))
    if _scored(case):
        pairs *= (1 - case["padding"] / max(case["T"], case["padding"] + 1)) / max(1, case["clips"]) * (0.55 if case["causal"] else 1)
    n = N * case["heads"] * case["dim"] * 2
    kept = 0.5 + 0.5 / GROUP
    tensors = {"fwd": 4, "step": 8, "checkpoint": 8 + 8 * kept}[case["way"]]
    return {"bytes": tensors * n + 4 * N * case["heads"], "flops": pairs * case["dim"] * (4 if case["way"] == "fwd" else 14)}


# --------------------------------------------------------------------------- definitions in 64 bits
def _pow2(k):
    """2^k in 64 bits, from its exponent bits (a power function may be off by a bit)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_8bit(x, fmt):
    """64-bit values of the 8-bit form: for each group the least k with max|x| <= qmax 2^k (k >= -127), then
    x 2^-k to the nearest code (ties to even): whole numbers, or 4 significant bits down to 2^-9."""
    c = x.shape[-1]
    out = x.new_empty(*x.shape[:-1], c)
    for a in range(0, c, GROUP):
        part = x[..., a:a + GROUP].double()
        top = part.abs().amax(-1, keepdim=True)
        k = torch.ceil(torch.log2(top / QMAX[fmt])).nan_to_num(0, 0, -127).clamp(min=-127)
        k = torch.where((k > -127) & (top <= QMAX[fmt] * _pow2(k - 1)), k - 1, k)
        k = torch.where(top > QMAX[fmt] * _pow2(k), k + 1, k)
        y = part / _pow2(k)
        if fmt == "int8":
            y = y.round()
        else:
            step = _pow2((torch.frexp(y)[1] - 4).clamp(min=-9))
            y = (y / step).round() * step
        out[..., a:a + GROUP] = torch.where(top.isfinite(), y * _pow2(k), math.nan)
    return out


def _exact_norm(case, s):
    x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
    out = {}
    if case["way"] == "bwd":
        mean, rstd = s["mean"].double(), s["rstd"].double()
    else:
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        out = dict(y=torch.addcmul(beta, (x - mean[:, None]) * rstd[:, None], gamma), mean=mean, rstd=rstd)
    if case["way"] != "fwd":
        if case["way"] == "step":
            x = _exact_8bit(x, case["fmt"])
        hat = (x - mean[:, None]) * rstd[:, None]
        dy, n = s["dy"].double(), case["channels"]
        g = dy * gamma
        inner = torch.einsum("rc,rc->r", g, hat)
        dx = rstd[:, None] * (g - (g.sum(1)[:, None] + hat * inner[:, None]) / n)
        out |= dict(dx=dx, dgamma=torch.einsum("rc,rc->c", dy, hat), dbeta=dy.sum(0))
    return out


def _exact_selection(case, s):
    """Block of each token and the selected blocks [heads, nb, nb], zone by zone and row by row."""
    T, H, W, heads, dim = (case[k] for k in ("T", "H", "W", "heads", "dim"))
    blk = np.zeros((T, H, W), dtype=np.int64)
    nb = m = 0
    for zt in range(0, T, 8):
        for zh in range(0, H, 8):
            for zw in range(0, W, 8):
                a, b, c = SHAPES[s["shape"][m]]
                m += 1
                for t in range(zt, zt + 8, a):
                    for h in range(zh, zh + 8, b):
                        for w in range(zw, zw + 8, c):
                            blk[t:t + a, h:h + b, w:w + c] = nb
                            nb += 1
    blk = torch.from_numpy(blk.reshape(-1)).to(DEV)
    one = torch.zeros(nb, len(blk), dtype=torch.float64, device=DEV)
    one[blk, torch.arange(len(blk), device=DEV)] = 1
    one /= one.sum(1, keepdim=True)
    chosen = np.zeros((heads, nb, nb), dtype=bool)
    limit = max(case["top_k"], int(math.floor(case["frac"] * nb)))
    for h in range(heads):
        z = ((one @ s["Q"][0, :, h].double()) @ (one @ s["K"][0, :, h].double()).T / math.sqrt(dim)).cpu().numpy()
        for i in range(nb):
            order = np.argsort(-z[i], kind="stable")
            p = np.exp(z[i][order] - z[i].max())
            need = int(np.searchsorted(np.cumsum(p / p.sum()), TOP_P)) + 1
            chosen[h, i, order[:min(max(need, case["top_k"]), limit, nb)]] = True
    return blk, torch.from_numpy(chosen).to(DEV)


def _exact_attn(case, s):
    N, heads, dim, way = case["T"] * case["H"] * case["W"], case["heads"], case["dim"], case["way"]
    blk, chosen = _exact_selection(case, s)
    pos = s["pos"][0].double()
    doc = s["doc"][0] if s["doc"] is not None else torch.zeros(N, dtype=torch.int32, device=DEV)
    names = ["O"] + (["dQ", "dK", "dV"] if way != "fwd" else [])
    out = {k: torch.zeros(1, N, heads, dim, dtype=torch.float64, device=DEV) for k in names}
    out["lse"] = torch.zeros(1, heads, N, dtype=torch.float64, device=DEV)
    rows = 4096
    for h in range(heads):
        q, k, v = (s[x][0, :, h].double() for x in "QKV")
        q2, k2, v2 = (_exact_8bit(x, case["fmt"]) for x in (q, k, v)) if way == "checkpoint" else (q, k, v)
        for a in range(0, N, rows):
            r = slice(a, min(N, a + rows))
            seen = chosen[h][blk[r]][:, blk] & (doc[r, None] == doc) & (doc >= 0)
            if case["causal"]:
                seen &= (pos <= pos[r, None]) | (pos < case["prefix"])

            def scores(q, k):
                x = q[r] @ k.T / math.sqrt(dim)
                t = torch.tanh(x / case["cap"]) if case["cap"] else None
                x = case["cap"] * t if case["cap"] else x
                if s["slopes"] is not None:
                    x = x - float(s["slopes"][h]) * (pos[r, None] - pos).abs()
                return t, x.masked_fill(~seen, -math.inf)

            t, x = scores(q, k)
            lse = torch.logsumexp(x, 1)
            some = torch.isfinite(lse)
            p = torch.exp(x - torch.where(some, lse, 0)[:, None])
            o = p @ v
            out["lse"][0, h, r], out["O"][0, r, h] = lse, o
            if way == "fwd":
                continue
            if way == "checkpoint":
                t, x = scores(q2, k2)
                p = torch.exp(x - torch.where(some, lse, 0)[:, None])
                o = _exact_8bit(o.bfloat16().double(), case["fmt"])
            do = s["dO"][0, r, h].double()
            ds = p * (do @ v2.T - (do * o).sum(1, keepdim=True)) / math.sqrt(dim)
            if t is not None:
                ds = ds * (1 - t * t)
            out["dV"][0, :, h] += p.T @ do
            out["dQ"][0, r, h] = ds @ k2
            out["dK"][0, :, h] += ds.T @ q2[r]
    return out


def exact(case, seed):
    if case["op"] == "norm":
        return _exact_norm(case, _norm_inputs(case, seed))
    if case["op"] == "pack":
        return _exact_8bit(_rows(case, _gen(seed), 1.0, 0.5).double(), case["fmt"])
    return _exact_attn(case, _attn_inputs(case, seed))
