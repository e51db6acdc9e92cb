"""In-place forms of the block norms that would overwrite what backward() starts from (host logic, no GPU)."""

import pytest
import torch

from dynamic_block_sparse_variance_b200 import packed, prism as P


def test_what_backward_starts_from_is_kept():
    x, y, other = (torch.zeros(6, 64) for _ in range(3))
    for args in ((x, None, None, x), (x, y, None, y), (x, y, y, None), (x, y, y, other), (x, y, other, y)):
        with pytest.raises(P.PrismError, match="must not take the place") as e:
            packed._keep(*args)
        assert e.value.code == P.PRISM_EINVAL
    # x is not needed beside y; x_out in its place is
    for args in ((x, None, None, None), (x, None, None, other), (x, y, x, other), (x, y, other, x), (x, y, None, None)):
        packed._keep(*args)
    none = torch.zeros(0, 64)
    packed._keep(none, None, None, none)
