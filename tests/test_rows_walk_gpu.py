"""Layer norm over so many rows that the resident grid walks them in several steps, the last one partly filled: ring slots
used again, reductions' parities, addresses carried from step to step, groups of rows.

Values are small whole numbers, so that every sum over a row or over the rows is a whole number below 2^24, exact in fp32
in any order: one row or channel left out, taken twice or stale shows.  Where a quotient comes in, the bounds count its
roundings: u = 2^-24, and for the variance the depth of its sum (a thread adds at most max(32, C / 256) of a row's
channels, 20 more additions join the threads)."""
import math

import pytest
import torch

from test_rows import DTYPES, P, U, close, value_of  # noqa: F401  (the fixture)

# (leading shape, channels, how the rows lie): at least two full steps of forward and backward, and a rest
SHAPES = [((150001,), 64, "plain"), ((100003,), 33, "plain"), ((10003, 8), 128, "fused"), ((30001, 3), 31, "fused"),
          ((7001,), 1024, "wide"), ((5003,), 1536, "plain"), ((22003,), 1001, "odd"), ((6001,), 2048, "plain"),
          ((1501,), 4104, "plain"), ((1501,), 5120, "wide"), ((2303,), 4097, "plain"), ((901,), 12288, "plain"),
          ((2401,), 16400, "plain")]


def place(lead, C, dtype, kind):
    if kind == "plain":
        return torch.empty(*lead, C, dtype=dtype, device="cuda")
    if kind == "wide":
        return torch.full((*lead, C + 24), 7.0, dtype=dtype, device="cuda")[..., :C]
    if kind == "odd":
        return torch.full((*lead, C + 5), 7.0, dtype=dtype, device="cuda")[..., 3:3 + C]
    return torch.full((lead[0], 3, *lead[1:], C), 7.0, dtype=dtype, device="cuda")[:, 1]


def whole(lead, C, dtype, kind, lo, hi, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = place(lead, C, dtype, kind)
    t.copy_(torch.randint(lo, hi + 1, (*lead, C), generator=g, device="cuda"))
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lead,C,kind", SHAPES)
def test_backward_over_many_rows(P, lead, C, kind, dtype):  # noqa: F811
    """With mean = 0 and rstd = 1 as the statistics, xhat is x: both weight gradients are exact, and so are the two sums
    over a row that dx needs (each channel's product at most 12 in size)."""
    t = DTYPES[dtype]
    x, dy = whole(lead, C, t, kind, -4, 4, 1), whole(lead, C, t, kind, -3, 3, 2)
    mean, rstd = torch.zeros(lead, device="cuda"), torch.ones(lead, device="cuda")
    X, D = x.double(), dy.double()
    dims = tuple(range(len(lead)))
    dgamma, dbeta = (D * X).sum(dims), D.sum(dims)
    assert max(dgamma.abs().max(), dbeta.abs().max()) < 2 ** 24
    a, b = D.mean(-1, keepdim=True), (D * X).mean(-1, keepdim=True)
    dx = D - a - X * b
    bound = 4 * U * (D.abs() + a.abs() + (X * b).abs())
    sources = [x] + [P.prism_ckpt_pack(x, f) for f in ("int8", "e4m3")]
    for k in sources[1:]:
        assert torch.equal(P.prism_ckpt_unpack(k), x)  # 8 bits hold these values exactly
    for src in sources:
        out = place(lead, C, t, kind)
        got = P.prism_layer_norm_bwd(dy, src, None, mean, rstd, dx=out)
        assert torch.equal(got[1].double(), dgamma) and torch.equal(got[2].double(), dbeta)
        close(out, dx, bound, "dx")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lead,C,kind", SHAPES)
def test_forward_over_many_rows(P, lead, C, kind, dtype):  # noqa: F811
    t = DTYPES[dtype]
    x = whole(lead, C, t, kind, 1, 9, 3)
    gamma = (1 + torch.arange(C, device="cuda") % 3).float()
    beta = (torch.arange(C, device="cuda") % 5).float()
    y, mean, rstd, kept = P.prism_layer_norm_fwd(x, gamma, beta, 1e-5, y=place(lead, C, t, kind), ckpt="int8")
    X = x.double()
    m = X.mean(-1)
    d = X - m[..., None]
    var = (d * d).mean(-1)
    r = (var + 1e-5).rsqrt()
    dm = 3 * U * m                                   # an exact sum times a rounded 1 / C
    n = max(32, math.ceil(C / 256)) + 20
    # a term (x - mean)^2 is off by 2 |d| (dm + u |d|) + u d^2, their sum by n u of itself
    dv = (n + 4) * U * var + 2 * dm * d.abs().mean(-1) + dm * dm
    dr = r * (dv / (var + 1e-5) / 2 + 4 * U)
    close(mean, m, dm, "mean")
    close(rstd, r, dr, "rstd")
    xhat = d * r[..., None]
    g, b = gamma.double(), beta.double()
    close(y, xhat * g + b, (d.abs() * dr[..., None] + (dm * r)[..., None] + 4 * U * xhat.abs()) * g + 3 * U * (xhat * g).abs() + 3 * U * b,
          "y")
    assert torch.equal(value_of(kept).reshape(X.shape), X.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("C", [1, 2, 7, 31, 32, 33, 64, 255, 257, 520, 1001, 1024, 2056, 4096, 4104, 8192, 8200, 12288, 12544, 16400,
                               36871])
def test_every_channel_counts_once(P, C, dtype):  # noqa: F811
    """Rows of 1, 2 and 3 with 96 in one channel, which moves through the first and last ones and the borders between
    threads, warps and the passes over a row: the mean is right to its last bits only if each channel is in it once."""
    t = DTYPES[dtype]
    at = sorted({c for b in (0, 8, 16, 32, 64, 256, 512, 1024, 2048, 4096, 8192, C // 2, C) for c in range(b - 9, b + 9)
                 if 0 <= c < C})
    x = (1 + torch.arange(C, device="cuda") % 3).to(t).expand(len(at), C).clone()
    x[torch.arange(len(at), device="cuda"), torch.tensor(at, device="cuda")] = 96
    _, mean, rstd = P.prism_layer_norm_fwd(x, eps=1e-5)
    m = x.double().mean(-1)
    close(mean, m, 3 * U * m, "mean")
    g = torch.zeros_like(x)
    g[torch.arange(len(at), device="cuda"), torch.tensor(at, device="cuda")] = 8
    one = torch.ones(len(at), device="cuda")
    # dx elsewhere is -mean(g) - x mean(g x) with mean 0 and rstd 1
    dx, dgamma, dbeta = P.prism_layer_norm_bwd(g, x, None, 0 * one, one)
    a, b = 8 / C, 8 * 96 / C
    want = g.double() - a - x.double() * b
    # (one channel: 8 - 8 - 96 * 768 = -73728, past fp16's 65504 and half a step: it rounds to -inf)
    past = want.abs() >= torch.finfo(t).max * (1 + torch.finfo(t).eps / 4)
    assert torch.equal(past, torch.full_like(past, C == 1 and dtype == "fp16")) and (dx[past] == -math.inf).all()
    close(dx[~past], want[~past], 4 * U * (g.double() + a + x.double() * b)[~past], "dx")
    hit = torch.zeros(C, dtype=torch.float64, device="cuda")
    hit[at] = 1
    assert torch.equal(dbeta.double(), 8 * hit) and torch.equal(dgamma.double(), 768 * hit)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lead,C,kind", [((200003,), 33, "plain"), ((30011,), 1001, "odd"), ((20011, 8), 128, "fused"),
                                         ((40009, 3), 40, "fused"), ((9001,), 4104, "wide"), ((301,), 70001, "odd"),
                                         ((65537,), 1024, "plain")])
def test_checkpoints_of_many_rows(P, lead, C, kind, dtype, fmt):  # noqa: F811
    """Rows are coded one by one: a tensor's codes, scales and values are those of its first, middle and last rows alone,
    which are few enough for one step (and whose codes test_rows.py compares with the definition)."""
    t = DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(4)
    x = place(lead, C, t, kind)
    x.copy_(torch.randn(*lead, C, generator=g, device="cuda") * torch.exp(3 * torch.randn(*lead, 1, generator=g, device="cuda")))
    k = P.prism_ckpt_pack(x, fmt)
    back = P.prism_ckpt_unpack(k, place(lead, C, t, kind))
    rows = math.prod(lead[1:])
    codes, scales = k.codes.view(lead[0], rows, C), k.scales.view(lead[0], rows, -1)
    for i in (0, lead[0] // 3, lead[0] // 2, lead[0] - 50):
        part = P.prism_ckpt_pack(x[i:i + 50].contiguous(), fmt)
        assert torch.equal(part.codes.view(50, rows, C), codes[i:i + 50])
        assert torch.equal(part.scales.view(50, rows, -1), scales[i:i + 50])
        assert torch.equal(P.prism_ckpt_unpack(part).nan_to_num(-1), back[i:i + 50].nan_to_num(-1))
    # and all of them: a value is off by at most half a step of its code and a rounding of its type.  int8: 2^(k-1) where
    # max|x| > 63.5 * 2^k, so below max / 127 of its group; e4m3: 2^-4 of itself.  (fp16 holds infinities here: their
    # groups read back as NaN.)
    top = torch.nn.functional.pad(x.float().abs(), (0, -C % 32)).unflatten(-1, (-1, 32)).amax(-1)
    top = top.repeat_interleave(32, -1)[..., :C]
    assert torch.equal(back.isnan(), top.isinf())
    off = (back.float() - x.float()).abs()
    allowed = top * ((1 / 127 if fmt == "int8" else 2.0 ** -4) + torch.finfo(t).eps)
    assert (off <= allowed + 2.0 ** -24)[top.isfinite()].all()
