"""Layer norm and 8-bit checkpoints: argument checks (no GPU) and the CUDA path
against the definitions in 64 bits.

u = 2^-24 is half a step of fp32.  A sum of n fp32 terms, in whatever order, is
off by at most (n - 1) u sum|terms| (to first order); a value rounded to type t
by eps(t) / 2 of itself.  The bounds below add these up with n = the longest
chain a row's or a column's sum can have (the row length, the row count), so they
hold for any summation order.
"""
import ctypes
import math

import pytest
import torch

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def P():
    from dynamic_block_sparse_zone_b200 import build as b
    b.build()
    import dynamic_block_sparse_zone_b200 as P
    P.load_library()
    return P


# --------------------------------------------------------------------------- no GPU
def _lib(P):
    from dynamic_block_sparse_zone_b200 import binding as B
    return B, P.load_library()


def test_row_arguments_are_checked_on_the_host(P):
    B, lib = _lib(P)
    at = lambda p, stride=64, gs=0, g=0: ctypes.byref(B.prism_rows(p, stride, gs, g))  # noqa: E731  never dereferenced
    k = lambda c=1 << 20, s=1 << 21, f=0: ctypes.byref(B.prism_ckpt(c, s, f))          # noqa: E731
    A, C = 1 << 24, 1 << 26

    def fwd(x=at(A), y=at(C), g=None, m=256, r=512, c=None, n=4, ch=64, eps=1e-6, dt=0, wdt=2):
        return lib.prism_layer_norm_fwd(x, g, None, y, m, r, c, n, ch, eps, dt, wdt, None)

    def says(word):
        assert word in lib.prism_last_error(), lib.prism_last_error()

    for kw, word in ((dict(x=None), b"x is NULL"), (dict(y=at(None)), b"y is NULL"), (dict(m=None), b"mean"),
                     (dict(n=-1), b"rows"), (dict(ch=0), b"channels"), (dict(ch=(1 << 20) + 1), b"channels"),
                     (dict(dt=3), b"dtype"), (dict(dt=0, wdt=1), b"weight_dtype"), (dict(eps=-1.0), b"eps"),
                     (dict(eps=float("nan")), b"eps"), (dict(x=at(A + 1)), b"aligned"), (dict(x=at(A, 63)), b"stride"),
                     (dict(x=at(A, 64, 10, 2)), b"group_stride"), (dict(x=at(A, 64, 64, -1)), b"group"),
                     (dict(y=at(A + 128)), b"overlap"), (dict(y=at(A, 64)), b"overlap"),
                     (dict(c=k(f=2)), b"format"), (dict(c=k(c=None)), b"checkpoint"), (dict(c=k(c=8)), b"aligned")):
        assert fwd(**kw) == 1, kw
        says(word)
    # the same buffer without shared elements: halves of wider rows; groups beside each other (sizes are
    # refused after the overlap check, so nothing is launched)
    assert fwd(x=at(A, 128), y=at(A + 127 * 2, 128)) == 1
    says(b"overlap")
    assert fwd(x=at(A, 128), y=at(A + 128, 128), c=k(f=7)) == 1
    says(b"format")
    assert fwd(x=at(A, 64, 384, 2), y=at(A + 256, 64, 384, 2), c=k(f=7)) == 1
    says(b"format")

    def bwd(x=at(A), c=None, dy=at(C), dx=at(1 << 28), dg=None, w=None, wb=0, n=4, ch=64):
        return lib.prism_layer_norm_bwd(x, c, dy, None, 256, 512, dx, dg, None, w, wb, n, ch, 0, 2, None)

    for kw, word in ((dict(x=None), b"exactly one"), (dict(c=k()), b"exactly one"), (dict(dx=at(C)), b"overlap"),
                     (dict(dx=at(A)), b"overlap"), (dict(dg=1024), b"workspace"),
                     (dict(dg=1024, w=4096, wb=8), b"needed"), (dict(dg=1024, w=4100, wb=1 << 20), b"workspace must be"),
                     (dict(x=None, c=k(f=9)), b"format")):
        assert bwd(**kw) == 1, kw
        says(word)
    assert lib.prism_ckpt_pack(None, 0, 4, 64, k(), None) == 1
    assert lib.prism_ckpt_pack(at(A), 0, 4, 64, None, None) == 1
    assert lib.prism_ckpt_unpack(None, at(A), 0, 4, 64, None) == 1
    assert lib.prism_ckpt_unpack(k(), at(A), 5, 4, 64, None) == 1
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.prism_ckpt_bytes(3, 65, ctypes.byref(a), ctypes.byref(b)) == 0 and (a.value, b.value) == (195, 9)
    assert lib.prism_ckpt_bytes(3, 0, ctypes.byref(a), ctypes.byref(b)) == 1
    assert lib.prism_layer_norm_bwd_workspace(-1, 64) == 0
    assert 0 < lib.prism_layer_norm_bwd_workspace(10 ** 6, 1 << 20) <= 64 << 20
    # nothing to do: no launch, no device needed
    assert fwd(n=0) == 0


def test_an_outputs_own_rows_are_checked(P):
    """Groups of an output that reach into one another are refused, and strides past any address; groups that follow one
    another or lie between one another's rows are not (what is refused then is the checkpoint's format, so nothing is
    launched)."""
    B, lib = _lib(P)
    A, C, D = 1 << 24, 1 << 30, 1 << 34
    at = lambda p, stride=64, gs=0, g=0: ctypes.byref(B.prism_rows(p, stride, gs, g))  # noqa: E731  never dereferenced
    bad_fmt = ctypes.byref(B.prism_ckpt(1 << 20, 1 << 21, 7))

    def fwd(y, x=at(A), n=12, k=bad_fmt):
        assert lib.prism_layer_norm_fwd(x, None, None, y, 256, 512, k, n, 64, 1e-6, 0, 2, None) == 1
        return lib.prism_last_error()

    assert b"reach into" in fwd(at(C, 64, 64, 4))         # groups of 4 rows, 64 elements apart
    assert b"reach into" in fwd(at(C, 128, 64, 4))
    assert b"reach into" in fwd(at(C, 64, 255, 4))
    assert b"reach into" in fwd(at(C, 191, 64, 4))        # three groups of 64 between rows 191 apart
    assert b"format" in fwd(at(C, 192, 64, 4))
    assert b"format" in fwd(at(C, 64, 256, 4))
    assert b"format" in fwd(at(C, 64, 64, 1))
    assert b"format" in fwd(at(C, 64, 64, 4), n=4)        # one group
    assert b"format" in fwd(at(C, 64, 256, 4), x=at(A, 64, 64, 4))  # an input may repeat rows
    assert b"address space" in fwd(at(C, 1 << 40), n=1 << 40)
    assert b"address space" in fwd(at(C, 64, 1 << 40, 4), n=1 << 30)
    assert lib.prism_layer_norm_bwd(at(A), None, at(C), None, 256, 512, at(D, 64, 64, 4), None, None, None, 0, 12, 64, 0, 2,
                                    None) == 1 and b"dx" in lib.prism_last_error()
    good = ctypes.byref(B.prism_ckpt(1 << 20, 1 << 21, 0))
    assert lib.prism_ckpt_unpack(good, at(D, 64, 64, 4), 0, 12, 64, None) == 1 and b"reach" in lib.prism_last_error()


def test_tensors_are_checked_by_the_binding(P):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        P.prism_layer_norm_fwd(x)  # not on a GPU
    with pytest.raises(ValueError):
        P.prism_ckpt_pack(x)


# --------------------------------------------------------------------------- GPU
def make(shape, dtype, seed, kind="plain"):
    """A CUDA tensor of `shape`: contiguous, a slice of wider rows, or heads of a fused projection."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "plain":
        t = torch.empty(shape, dtype=dtype, device="cuda")
    elif kind == "wide":
        t = torch.full((*shape[:-1], shape[-1] + 24), 7.0, dtype=dtype, device="cuda")[..., :shape[-1]]
    elif kind == "odd":
        t = torch.full((*shape[:-1], shape[-1] + 5), 7.0, dtype=dtype, device="cuda")[..., 3:3 + shape[-1]]
    else:  # fused: [tokens, heads, channels] inside [tokens, 3, heads, channels]
        t = torch.full((shape[0], 3, *shape[1:]), 7.0, dtype=dtype, device="cuda")[:, 1]
    t.copy_(torch.randn(shape, generator=g, device="cuda") * (1 + torch.arange(shape[-1], device="cuda") % 5) + 0.5)
    return t


def value_of(ckpt):
    """A checkpoint's values from its bytes, in 64 bits on the CPU."""
    codes, scales = ckpt.codes.cpu(), ckpt.scales.cpu().double()
    q = codes.view(torch.int8).double() if ckpt.format == "int8" else codes.view(torch.float8_e4m3fn).double()
    s = torch.where(scales == 255, math.nan, torch.pow(torch.tensor(2.0, dtype=torch.float64), scales - 127))
    return q * s.repeat_interleave(32, 1)[:, :codes.shape[1]]


def reference_8bit(x, fmt):
    """The definition on the CPU in 64 bits: (values, exponents) of x [rows, channels]."""
    x = x.detach().cpu().double()
    rows, C = x.shape
    pad = torch.nn.functional.pad(x, (0, -C % 32)).reshape(rows, -1, 32)
    qmax = 127.0 if fmt == "int8" else 448.0
    top = pad.abs().amax(2)
    k = torch.full(top.shape, -127.0, dtype=torch.float64)
    for e in range(-126, 129):
        k = torch.where(top > qmax * 2.0 ** (e - 1), float(e), k)
    q = pad / 2.0 ** k[..., None]
    if fmt == "int8":
        q = q.round()
    else:
        step = 2.0 ** (torch.frexp(q)[1].double() - 4).clamp(min=-9)
        q = (q / step).round() * step
    v = torch.where(top[..., None].isfinite(), q * 2.0 ** k[..., None], math.nan)
    return v.reshape(rows, -1)[:, :C], k


SHAPES = [((1, 1), "plain"), ((1, 1024), "plain"), ((3, 31), "plain"), ((5, 33), "odd"), ((257, 64), "plain"),
          ((40, 8, 128), "fused"), ((7, 5, 96), "fused"), ((33, 1000), "wide"), ((130, 1001), "odd"), ((64, 1536), "plain"),
          ((9, 2048), "wide"), ((5, 4104), "plain"), ((3, 10007), "plain"), ((2, 40000), "plain"), ((1, 70001), "odd")]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape,kind", SHAPES)
def test_checkpoint_codes_are_the_definition(P, shape, kind, dtype, fmt):
    x = make(shape, DTYPES[dtype], 1, kind)
    k = P.prism_ckpt_pack(x, fmt)
    flat = x.reshape(-1, shape[-1])
    want, e = reference_8bit(flat, fmt)
    assert torch.equal(k.scales.cpu().double() - 127, e)
    assert torch.equal(value_of(k), want)
    back = P.prism_ckpt_unpack(k)
    assert back.shape == x.shape and back.dtype == x.dtype
    assert torch.equal(back.reshape(want.shape).cpu().double(), want.to(DTYPES[dtype]).double())
    out = make(shape, DTYPES[dtype], 2, kind)
    assert torch.equal(P.prism_ckpt_unpack(k, out), back)
    if kind != "plain":  # what lies between the rows is left alone
        whole = out.as_strided((out.untyped_storage().nbytes() // out.element_size(),), (1,), 0)
        mask = torch.ones_like(whole, dtype=torch.bool)
        mask.as_strided(out.shape, out.stride(), out.storage_offset())[...] = False
        assert (whole[mask] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_checkpoint_extremes(P, dtype, fmt):
    t = DTYPES[dtype]
    top, tiny = torch.finfo(t).max, torch.finfo(t).smallest_normal
    x = torch.zeros(12, 64, dtype=t, device="cuda")
    x[1, 3], x[2, 40], x[3, 5] = math.inf, -math.inf, math.nan     # that group reads back as NaN, its neighbour does not
    x[:4, 63] = 3.0
    x[1, 63] = x[1, 40] = 5.0
    x[4], x[5], x[6] = top, -top, tiny
    x[7, ::2] = tiny / 4                                            # below the normal range
    x[8, 0], x[8, 1:] = 1.0, -0.0
    x[9, :32], x[9, 32:] = 127.0, 448.0                             # exactly qmax
    x[10, :32], x[10, 32:] = 127.5, 449.0
    x[11] = torch.linspace(-1, 1, 64, dtype=torch.float32, device="cuda").to(t)
    k = P.prism_ckpt_pack(x, fmt)
    want, _ = reference_8bit(x, fmt)
    assert torch.equal(torch.nan_to_num(value_of(k), nan=1e300), torch.nan_to_num(want, nan=1e300))
    back = P.prism_ckpt_unpack(k).cpu().double()
    limited = want.clamp(-top, top)                                 # a code may stand for a little more than the largest
    limited = torch.where(want.isnan(), math.nan, limited).to(t).double()
    assert torch.equal(torch.nan_to_num(back, nan=1e300), torch.nan_to_num(limited, nan=1e300))
    assert back[1, :32].isnan().all() and back[2, 32:].isnan().all() and back[3, :32].isnan().all()
    assert back[1, 32:].isfinite().all() and back[4].isfinite().all()


def norm_fwd_reference(x, gamma, beta, eps):
    x = x.double()
    C = x.shape[-1]
    mean = x.mean(-1)
    d = x - mean[..., None]
    var = (d * d).mean(-1)
    rstd = 1 / (var + eps).sqrt()
    xhat = d * rstd[..., None]
    g = torch.ones(C, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros(C, dtype=torch.float64, device=x.device) if beta is None else beta.double()
    y = xhat * g + b
    n = C + 4
    dmean = n * U * x.abs().mean(-1)
    # var's terms carry (x - mean)'s errors: 2|d| (dmean + u|d|) each
    dvar = n * U * var + 2 * dmean * d.abs().mean(-1) + 2 * U * var + dmean ** 2
    drstd = rstd * (dvar / (var + eps) / 2 + 4 * U)
    dhat = d.abs() * drstd[..., None] + (dmean * rstd)[..., None] + 3 * U * xhat.abs()
    dy = dhat * g.abs() + 3 * U * (y.abs() + b.abs())
    return (y, mean, rstd), (dy, dmean, drstd)


def norm_bwd_reference(x, dy, gamma, mean, rstd):
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[..., None], rstd.double()[..., None]
    C = x.shape[-1]
    g = dy * (torch.ones(C, dtype=torch.float64, device=x.device) if gamma is None else gamma.double())
    xhat = (x - mean) * rstd
    a, b = g.mean(-1, keepdim=True), (g * xhat).mean(-1, keepdim=True)
    dx = rstd * (g - a - xhat * b)
    n = C + 4
    # x - mean is rounded to u of itself, and is as large as xhat / rstd
    dhat = 3 * U * xhat.abs()
    da = n * U * g.abs().mean(-1, keepdim=True)
    db = (n + 4) * U * (g * xhat).abs().mean(-1, keepdim=True)
    ddx = rstd * (4 * U * (g.abs() + a.abs() + (xhat * b).abs()) + da + xhat.abs() * db + dhat * b.abs()) + 2 * U * dx.abs()
    lead = tuple(range(x.dim() - 1))
    rows = math.prod(x.shape[:-1])
    dgamma, dbeta = (dy * xhat).sum(lead), dy.sum(lead)
    return (dx, dgamma, dbeta), (ddx, (rows + 4) * U * (dy * xhat).abs().sum(lead), (rows + 4) * U * dy.abs().sum(lead))


def close(got, want, bound, what):
    """|got - want| <= bound + half a step of got's type at want (and of its smallest normal)."""
    f = torch.finfo(got.dtype)
    allowed = bound + f.eps / 2 * (want.abs() + bound) + f.smallest_normal * f.eps
    off = (got.double() - want).abs()
    assert (off <= allowed).all(), f"{what}: {(off - allowed).max().item():.3e} over the bound, off {off.max().item():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["fp32", "own", "none"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape,kind", SHAPES)
def test_layer_norm_forward_and_backward(P, shape, kind, dtype, weights):
    t = DTYPES[dtype]
    C = shape[-1]
    x, dy = make(shape, t, 3, kind), make(shape, t, 4, kind)
    wt = torch.float32 if weights == "fp32" else t
    g = torch.Generator(device="cuda").manual_seed(5)
    gamma = None if weights == "none" else (1 + 0.3 * torch.randn(C, generator=g, device="cuda")).to(wt)
    beta = None if weights == "none" else torch.randn(C, generator=g, device="cuda").to(wt)
    y, mean, rstd = P.prism_layer_norm_fwd(x, gamma, beta, 1e-5)
    (ry, rm, rr), (by, bm, br) = norm_fwd_reference(x, gamma, beta, 1e-5)
    close(mean, rm, bm, "mean")
    close(rstd, rr, br, "rstd")
    close(y, ry, by, "y")
    dx, dgamma, dbeta = P.prism_layer_norm_bwd(dy, x, gamma, mean, rstd)
    want, bound = norm_bwd_reference(x, dy, gamma, mean, rstd)
    for got, w, b, what in zip((dx, dgamma, dbeta), want, bound, ("dx", "dgamma", "dbeta")):
        close(got, w, b, what)
    again = P.prism_layer_norm_bwd(dy, x, gamma, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dgamma, dbeta)))
    only = P.prism_layer_norm_bwd(dy, x, gamma, mean, rstd, weight_grads=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    out = make(shape, t, 6, kind)  # written in place among other elements
    assert P.prism_layer_norm_bwd(dy, x, gamma, mean, rstd, dx=out)[0] is out and torch.equal(out, dx)
    assert torch.equal(P.prism_layer_norm_fwd(x, gamma, beta, 1e-5, y=out)[0], y)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape,kind", SHAPES)
def test_layer_norm_through_a_checkpoint(P, shape, kind, dtype, fmt):
    t = DTYPES[dtype]
    x, dy = make(shape, t, 7, kind), make(shape, t, 8, "plain")
    gamma = torch.linspace(0.5, 1.5, shape[-1], device="cuda")
    y, mean, rstd, kept = P.prism_layer_norm_fwd(x, gamma, None, 1e-6, ckpt=fmt)
    assert all(torch.equal(a, b) for a, b in zip((y, mean, rstd), P.prism_layer_norm_fwd(x, gamma, None, 1e-6)))
    alone = P.prism_ckpt_pack(x, fmt)
    assert torch.equal(kept.codes, alone.codes) and torch.equal(kept.scales, alone.scales)
    xq = value_of(kept).reshape(shape).cuda()
    want, bound = norm_bwd_reference(xq, dy, gamma, mean, rstd)
    for got, w, b, what in zip(P.prism_layer_norm_bwd(dy, kept, gamma, mean, rstd), want, bound, ("dx", "dgamma", "dbeta")):
        close(got, w, b, what)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_channel_counts_in_turn(P, dtype):
    """Every way a row is laid over threads, small to large and back: a kernel's shared memory grows with the channels."""
    t = DTYPES[dtype]
    sizes = [8, 72, 256, 520, 768, 1024, 1280, 1536, 2048, 2056, 3328, 4096, 6144, 8184, 8192, 8200, 11264, 12288, 12544,
             13312, 16384, 16400, 17408, 24576, 32768, 33000, 257, 511, 1023, 1027, 2049, 4095, 4097, 8191, 8193]
    for C in sizes + sizes[::-1]:
        x, dy = make((5, C), t, C), make((5, C), t, C + 1)
        gamma = torch.linspace(0.5, 1.5, C, device="cuda")
        y, mean, rstd, kept = P.prism_layer_norm_fwd(x, gamma, gamma, 1e-5, ckpt="int8")
        (ry, rm, rr), (by, bm, br) = norm_fwd_reference(x, gamma, gamma, 1e-5)
        close(y, ry, by, f"y {C}")
        close(rstd, rr, br, f"rstd {C}")
        for src in (x, kept):
            want, bound = norm_bwd_reference(x if src is x else value_of(kept).cuda(), dy, gamma, mean, rstd)
            for got, w, b, what in zip(P.prism_layer_norm_bwd(dy, src, gamma, mean, rstd), want, bound, ("dx", "dgamma", "dbeta")):
                close(got, w, b, f"{what} {C}")


@pytest.mark.gpu
def test_layer_norm_gradient_against_differences(P):
    """d(sum y w)/d(x, gamma, beta) by central differences of the 64-bit definition."""
    x, w = make((6, 48), torch.float32, 9), make((6, 48), torch.float32, 10)
    gamma = torch.linspace(0.5, 1.5, 48, device="cuda")
    beta = torch.linspace(-1, 1, 48, device="cuda")
    _, mean, rstd = P.prism_layer_norm_fwd(x, gamma, beta, 1e-3)
    got = P.prism_layer_norm_bwd(w, x, gamma, mean, rstd)
    loss = lambda x, g, b: (norm_fwd_reference(x, g, b, 1e-3)[0][0] * w.double()).sum()  # noqa: E731
    h = 1e-5
    args = [x.double(), gamma.double(), beta.double()]
    for i, grad in enumerate(got):
        flat = args[i].reshape(-1)
        for j in range(0, flat.numel(), 7):
            up, down = flat.clone(), flat.clone()
            up[j] += h
            down[j] -= h
            vals = [loss(*[a if m != i else v.reshape(a.shape) for m, a in enumerate(args)]) for v in (up, down)]
            # the difference's own error is O(h^2) of the third derivative: under 1e-6 at these sizes;
            # fp32 sums of 48 terms of up to ~30 are off by under 1e-4
            assert abs((vals[0] - vals[1]) / (2 * h) - grad.reshape(-1)[j]) < 2e-4


@pytest.mark.gpu
@pytest.mark.parametrize("channels", [1, 8, 64, 1000, 40000])
def test_no_rows(P, channels):
    x = torch.empty(0, channels, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(channels, device="cuda")
    y, mean, rstd, kept = P.prism_layer_norm_fwd(x, gamma, gamma, ckpt="int8")
    assert y.shape == x.shape and mean.numel() == 0 and kept.codes.numel() == 0
    dx, dgamma, dbeta = P.prism_layer_norm_bwd(x, x, gamma, mean, rstd)
    assert dx.shape == x.shape and (dgamma == 0).all() and (dbeta == 0).all()
    assert P.prism_layer_norm_bwd(x, kept, gamma, mean, rstd)[1].eq(0).all()
    assert P.prism_ckpt_unpack(kept).shape == x.shape


@pytest.mark.gpu
def test_constant_rows_and_large_offsets(P):
    x = torch.full((3, 777), 4.0, device="cuda")
    y, mean, rstd = P.prism_layer_norm_fwd(x, eps=1e-6)
    # the fp32 mean of equal values is off by at most 777 u 4, and rstd <= 1000
    assert (y.abs() <= 777 * U * 4 * 1000).all() and (rstd <= 1000.001).all()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(5, 2048, generator=g, device="cuda") + 1000.0
    (ry, rm, rr), (by, bm, br) = norm_fwd_reference(x, None, None, 1e-6)
    y, mean, rstd = P.prism_layer_norm_fwd(x)
    close(mean, rm, bm, "mean")
    close(rstd, rr, br, "rstd")
    close(y, ry, by, "y")


@pytest.mark.gpu
def test_a_nan_stays_in_its_row(P):
    x = make((9, 520), torch.bfloat16, 11)
    dy = make((9, 520), torch.bfloat16, 12)
    clean = P.prism_layer_norm_fwd(x)
    x2 = x.clone()
    x2[4, 17] = math.nan
    y, mean, rstd = P.prism_layer_norm_fwd(x2)
    keep = [r for r in range(9) if r != 4]
    assert y[4].isnan().all() and torch.equal(y[keep], clean[0][keep])
    dx = P.prism_layer_norm_bwd(dy, x2, None, mean, rstd)[0]
    assert dx[4].isnan().all() and torch.equal(dx[keep], P.prism_layer_norm_bwd(dy, x, None, *clean[1:])[0][keep])


@pytest.mark.gpu
def test_streams_graphs_and_overlapping_calls(P):
    """Calls on two streams at once, and a captured step replayed on new inputs."""
    x = [make((2000, 1024), torch.bfloat16, s) for s in (20, 21)]
    dy = [make((2000, 1024), torch.bfloat16, s) for s in (22, 23)]
    gamma = torch.linspace(0.5, 1.5, 1024, device="cuda")

    def step(x, dy):
        y, mean, rstd, kept = P.prism_layer_norm_fwd(x, gamma, gamma, ckpt="e4m3")
        return (y, *P.prism_layer_norm_bwd(dy, kept, gamma, mean, rstd))

    alone = [step(a, b) for a, b in zip(x, dy)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        both = []
        for s, a, b in zip(streams, x, dy):
            with torch.cuda.stream(s):
                both.append(step(a, b))
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            assert all(torch.equal(p, q) for p, q in zip(got, want))
    xin, din = x[0].clone(), dy[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(xin, din)
    xin.copy_(x[1])
    din.copy_(dy[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, alone[1]))


@pytest.mark.gpu
def test_refusals_of_the_binding(P):
    x = make((4, 64), torch.bfloat16, 30)
    gamma = torch.ones(64, device="cuda")
    y, mean, rstd, kept = P.prism_layer_norm_fwd(x, gamma, ckpt="int8")
    bad = [lambda: P.prism_layer_norm_fwd(x.t()), lambda: P.prism_layer_norm_fwd(x, gamma[:32]),
           lambda: P.prism_layer_norm_fwd(x, gamma.double()), lambda: P.prism_layer_norm_fwd(x, gamma, gamma.bfloat16()),
           lambda: P.prism_layer_norm_fwd(x.double()), lambda: P.prism_layer_norm_fwd(x, gamma, ckpt="fp4"),
           lambda: P.prism_layer_norm_fwd(x[:1].expand(4, 64)), lambda: P.prism_layer_norm_fwd(x, y=x[:2]),
           lambda: P.prism_layer_norm_bwd(x, kept, gamma, mean[:2], rstd), lambda: P.prism_layer_norm_bwd(x[:2], kept, gamma, mean, rstd),
           lambda: P.prism_layer_norm_bwd(x, x.float(), gamma, mean, rstd), lambda: P.prism_ckpt_pack(x, "int4"),
           lambda: P.prism_ckpt_unpack(kept, x[:2]), lambda: P.prism_layer_norm_bwd(x, kept, gamma, mean.cpu(), rstd)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(P.PrismError, match="overlap"):
        P.prism_layer_norm_fwd(x, y=x)
    with pytest.raises(P.PrismError, match="overlap"):
        P.prism_layer_norm_bwd(x, kept, gamma, mean, rstd, dx=x)
