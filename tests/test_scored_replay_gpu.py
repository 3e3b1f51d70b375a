"""Captured scored passes, replayed after the plan has changed behind the host's checks: under scores of the same kind
they compute with the current ones, under others (or none) they leave their outputs and the plan's tensors alone and the
plan's check says so."""
import numpy as np
import pytest
import torch

from test_scored_gpu import SHAPES, Case, P  # noqa: F401  (the fixture)

MARK = 7.0


class Captured:
    def __init__(self, c, checkpoint=False):
        self.c = c
        self.outs = [torch.empty_like(c.Q) for _ in range(4)]
        self.O0 = c.plan.fwd(scored=True)[0]
        kept = c.plan.save(c.Q, c.K, c.V, *c.plan.fwd(scored=True)) if checkpoint else None
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            c.plan.fwd(self.outs[0], scored=True, want_lse=False)
            if checkpoint:
                c.plan.bwd_ckpt(kept, c.dO, *self.outs[1:], scored=True)
            else:
                c.plan.bwd(self.outs[0], c.dO, *self.outs[1:], scored=True)

    def replay(self):
        for x in self.outs:
            x.fill_(MARK)
        self.graph.replay()
        torch.cuda.synchronize()
        return self.outs

    def refused(self, P):  # noqa: F811
        O, dQ, dK, dV = self.replay()
        assert all((x == MARK).all() for x in (O, dK, dV)) and (dQ == 0).all()
        with pytest.raises(P.PrismError, match="ERR_STATE.*other scores"):
            self.c.plan.check()
        self.c.plan.check()  # said once

    def runs(self):
        got = [x.clone() for x in self.replay()]
        self.c.plan.check()
        O, _ = self.c.plan.fwd(scored=True)
        dQ, dK, dV = self.c.plan.bwd(O, self.c.dO, scored=True)
        torch.cuda.synchronize()
        assert torch.equal(got[0], O) and torch.equal(got[2], dK) and torch.equal(got[3], dV)
        # dQ's partial sums are added in the order they arrive
        assert (got[1].float() - dQ.float()).abs().max() <= 2.0 ** -8 * dQ.float().abs().max()


def rebuild(c, seed):
    """The same tensors under other zone shapes: other blocks, lists, permutation."""
    shape = np.random.default_rng(seed).integers(0, len(SHAPES), (c.batch, c.N // 512)).astype(np.int32)
    c.plan.build_with_zones(c.Q, c.K, c.V, np.vectorize(lambda i: int(np.prod(SHAPES[i])))(shape), shape)


@pytest.mark.gpu
@pytest.mark.parametrize("form", [dict(cap=10.0), dict(clips=2, padding=3, causal=True, slope=0.2)])
@pytest.mark.parametrize("dim", [64, 128])
def test_behind_another_build(P, dim, form):  # noqa: F811
    c = Case(P, 16, 16, 8, 2, dim, seed=50, **form)
    kw = dict(cap=c.cap, slopes=c.slopes, doc=c.doc, causal=c.causal)
    t = Captured(c)
    t.runs()
    rebuild(c, 51)
    sparse = c.plan.fwd()[0]
    t.refused(P)
    assert torch.equal(c.plan.fwd()[0], sparse)  # no row of the plan's Q, K, V was taken for padding
    c.plan.set_score(**kw)
    t.runs()
    rebuild(c, 52)
    t.refused(P)
    c.plan.close()


@pytest.mark.gpu
def test_under_other_scores(P):  # noqa: F811
    c = Case(P, 16, 16, 8, 2, 64, cap=10.0, seed=53)
    t = Captured(c)
    doc = (torch.arange(c.N, device="cuda") // 700).int()[None]
    for kw in (dict(cap=11.0), dict(), dict(cap=10.0, causal=True), dict(cap=10.0, doc=doc),
               dict(cap=10.0, slopes=torch.ones(2, device="cuda"))):
        c.plan.update_qkv(c.Q, c.K, c.V)
        c.plan.set_score(**kw)
        t.refused(P)
    c.plan.update_qkv(c.Q, c.K, c.V)
    c.plan.set_score(cap=10.0)
    t.runs()
    c.plan.close()


@pytest.mark.gpu
def test_under_other_documents_and_positions(P):  # noqa: F811
    """Packed batches: the step is captured once, the scores are set by hand for each batch."""
    c = Case(P, 16, 16, 8, 2, 64, clips=2, causal=True, slope=0.3, cap=9.0, seed=54)
    t = Captured(c)
    for cut in (300, 1111, 2047):
        n = torch.arange(c.N, device="cuda")
        doc = torch.where(n < cut, 0, 1).int()[None]
        doc[:, -40:] = -1
        pos = torch.where(n < cut, n, n - cut).float()[None]
        c.plan.update_qkv(c.Q, c.K, c.V)
        c.plan.set_score(cap=9.0, slopes=c.slopes * cut / 1000, pos=pos, doc=doc, causal=True)
        t.runs()
    c.plan.close()


@pytest.mark.gpu
def test_a_scored_backward_from_a_checkpoint(P):  # noqa: F811
    c = Case(P, 16, 16, 8, 2, 64, clips=3, padding=2, seed=55)
    t = Captured(c, checkpoint=True)
    rebuild(c, 56)
    t.refused(P)
    c.plan.close()


@pytest.mark.gpu
def test_a_reported_timeout_leaves_the_scores(P):  # noqa: F811
    c = Case(P, 8, 16, 16, 2, 64, cap=10.0, clips=2, seed=57)
    want = c.run()
    c.plan.selftest_timeout()
    with pytest.raises(P.PrismError, match="ERR_TIMEOUT"):
        c.plan.check()
    got = c.run()  # checks the plan
    assert torch.equal(got["O"], want["O"]) and torch.equal(got["dV"], want["dV"])
    c.plan.close()
