"""Key offsets that run backwards are seen where there are no queries too: only the kind of CTA that keeps dK and dV
runs then, and the search for a slot's sequence passes such a sequence by."""

import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.packed import PackedAttention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad,used", [([0, 200, 100, 300], None), ([0, 100, 100, 301], None), ([0, 100, 250, 300], [100, 151, 50])])
def test_bad_key_offsets_without_queries_are_latched(bad, used):
    ints = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
    q, k = (torch.ones(n, 2, 64, dtype=torch.bfloat16, device="cuda") for n in (0, 300))
    att = PackedAttention(2, 2, 64)
    o = att.forward(q, k, k, ints([0, 0, 0, 0]), ints(bad), k_used=None if used is None else ints(used))
    P.prism_device_status()
    att.backward(o)
    with pytest.raises(P.PrismError) as e:
        P.prism_device_status()
    assert e.value.code == P.PRISM_EBOUNDS
    att.forward(q, k, k, ints([0, 0, 0, 0]), ints([0, 100, 250, 300]))
    assert all((g == 0).all() for g in att.backward(o))
    P.prism_device_status()
