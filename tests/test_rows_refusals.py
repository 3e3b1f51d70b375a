"""Refusals of the row operators' binding that need no memory behind the tensors (no GPU)."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


def test_groups_too_long_for_the_c_interface_are_refused():
    """A group of 2^32 rows came out as group = 0 (32 bits), which means evenly spaced rows."""
    from dynamic_block_sparse_zone_b200 import binding as B
    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")  # a fake tensor's address is 0
        wide = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda:0")  # noqa: E731
        for rows in (2 ** 32, 2 ** 32 + 4, 2 ** 31):
            with pytest.raises(ValueError, match="groups"):
                B._rows(wide(2, 2 * rows, 2)[:, :rows, :1], "x")
        with pytest.raises(ValueError, match="groups"):
            B._rows(wide(2 ** 30, 4, 2)[:, :3, :1], "x")           # 3 * 2^30 rows in all
        r, n, C = B._rows(wide(2, 2 ** 30, 2)[:, :2 ** 29, :1], "x")
        assert (r.group, r.stride, r.group_stride, n, C) == (2 ** 29, 2, 2 ** 31, 2 ** 30, 1)
        r, n, _ = B._rows(wide(2 ** 33, 2)[:, :1], "x")            # evenly spaced: any number
        assert (r.group, r.stride, n) == (0, 2, 2 ** 33)
