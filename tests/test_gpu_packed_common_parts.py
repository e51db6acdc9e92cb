"""Keys and values with a part that is common to all of them, as projections with a bias give: the softmax does not
see a common part of the keys, and an average of values with a common part is that part plus the rest's average.
What the rounding of the probabilities does must not be multiplied by either."""

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.packed import PackedAttention
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _f64(t):
    return t.detach().double().cpu().numpy()


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# lengths of queries and keys, heads, kv heads: single tiles, pairs of tiles, split keys, the 16-row kernel whole and split
SHAPES = [([90, 3, 200], [90, 40, 200], 4, 2), ([700], [700], 2, 1), ([130], [1500], 2, 2), ([3, 2], [100, 77], 4, 2),
          ([1], [2000], 8, 2)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lq,lk,heads,kv", SHAPES)
def test_an_average_of_equal_values_is_that_value(lq, lk, heads, kv, dim):
    """With v the same in every row O is v: the weights that form it and their sum carry the same roundings. What is
    left is the sums in 32 bits: up to 2000 terms, 2^-24 each in any order below 2^-13 of the value, and a split
    adds two more roundings. O and its residual together have 16 bits, so the test sees it."""
    gen = torch.Generator().manual_seed(dim + lk[0])
    qo, ko = ref.offsets(lq), ref.offsets(lk)
    q = (torch.randn(qo[-1], heads, dim, generator=gen) * 1.5).to(BF16).cuda()
    k = (torch.randn(ko[-1], kv, dim, generator=gen) * 1.5).to(BF16).cuda()
    v = torch.randn(1, kv, dim, generator=gen).to(BF16).cuda().expand(int(ko[-1]), kv, dim).contiguous()
    p = P.prism_packed_params(seqs=len(lq), heads=heads, kv_heads=kv, head_dim=dim, q_rows=int(qo[-1]), k_rows=int(ko[-1]),
                              causal=1)
    o, res = (torch.empty_like(q) for _ in range(2))
    lse = torch.empty(heads, int(qo[-1]), device="cuda")
    ws = torch.empty(P.prism_packed_workspace_size(p, P.PRISM_WS_PACKED_FWD), dtype=torch.uint8, device="cuda")
    P.prism_packed_attn_fwd(p, q, k, v, _ints(qo), _ints(ko), None, o, res, lse, ws)
    P.prism_device_status()
    want = _f64(v[:1].repeat_interleave(heads // kv, 1))
    seen = np.isfinite(lse.T.cpu().numpy())
    err = np.abs(_f64(o) + _f64(res) - want)[seen]
    assert seen.any() and (err <= (2.0 ** -13 + 2.0 ** -16) * np.broadcast_to(np.abs(want), o.shape)[seen]).all(), err.max()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("k_common,v_common", [(0.0, 13.0), (13.0, 0.0), (13.0, 13.0)])
@pytest.mark.parametrize("lq,lk,heads,kv", [([600], [600], 2, 2), ([300, 37, 500], [300, 90, 500], 4, 2), ([60], [60], 6, 2),
                                           ([3, 2], [1000, 770], 4, 2), ([9], [2000], 8, 2)])
def test_gradients_beside_common_parts(lq, lk, heads, kv, k_common, v_common, dim, causal):
    """A row of dS = P (dP - D) sums to zero, so dQ = scale dS K has nothing of the keys' common part, and D takes the
    values' out of dP. Three independent roundings (the operand dS, P inside D, the result), each of a mean square of
    at most U^2 / 3 of what varies: U of the norm. A rounding that meets a common part of 13 times the rest's size
    instead gives up to 13 times that for either part (and 13 x 13 for both)."""
    gen = torch.Generator().manual_seed(int(k_common + 2 * v_common) + dim)
    qo, ko = ref.offsets(lq), ref.offsets(lk)
    r = lambda *s: torch.randn(*s, generator=gen)
    q, dout = (r(int(qo[-1]), heads, dim).to(BF16).cuda() for _ in range(2))
    k = (r(int(ko[-1]), kv, dim) + k_common * r(1, kv, dim)).to(BF16).cuda()
    v = (r(int(ko[-1]), kv, dim) + v_common * r(1, kv, dim)).to(BF16).cuda()
    att = PackedAttention(heads, kv, dim, causal=causal)
    o = att.forward(q, k, v, _ints(qo), _ints(ko))
    grads = dict(zip(("dq", "dk", "dv"), att.backward(dout)))
    P.prism_device_status()
    want, _, _ = ref.attention(_f64(q), _f64(k), _f64(v), qo, ko, causal, dim ** -0.5, None, _f64(dout))
    for n, g in (("o", o), *grads.items()):
        err = np.linalg.norm(_f64(g) - want[n])
        assert err <= ref.U * np.linalg.norm(want[n]), f"{n}: {err / np.linalg.norm(want[n]):.2e}"
