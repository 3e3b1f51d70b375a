"""Scored passes refuse tensors of another device than the current one.  (One GPU: what the calls are given only says
that it lies elsewhere, and is never read.)"""
from types import SimpleNamespace

import pytest
import torch

from test_scored_gpu import Case, P  # noqa: F401  (the fixture)


def away(t):
    return SimpleNamespace(is_cuda=True, dtype=t.dtype, shape=t.shape, is_contiguous=lambda: True,
                           device=torch.device("cuda", torch.cuda.current_device() + 1))


@pytest.mark.gpu
def test_scored_passes_refuse_tensors_of_another_device(P):  # noqa: F811
    c = Case(P, 8, 16, 16, 2, 64, cap=10.0, seed=41)
    with pytest.raises(ValueError, match="O is on cuda"):
        c.plan.fwd(away(c.Q), scored=True)
    with pytest.raises(ValueError, match="lse is on cuda"):
        c.plan.fwd(lse=away(torch.empty(1, 2, c.N)), scored=True)
    O, _ = c.plan.fwd(scored=True)
    for name in ("O", "dO", "dQ", "dK", "dV"):
        args = {**dict(O=O, dO=c.dO), name: away(O)}
        with pytest.raises(ValueError, match=f"{name} is on cuda"):
            c.plan.bwd(**args, scored=True)
    c.plan.bwd(O, c.dO, scored=True)
    torch.cuda.synchronize()
    c.plan.close()
