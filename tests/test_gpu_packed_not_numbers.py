"""A NaN that a row sees shows in that row, whichever kernel runs and however the keys are split, and in no other."""

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.packed import PackedAttention
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN = float("nan")


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _inputs(lq, lk, heads, kv, dim):
    gen = torch.Generator().manual_seed(dim + sum(lk))
    r = lambda n, h: torch.randn(n, h, dim, generator=gen).to(BF16).cuda()
    return r(sum(lq), heads), r(sum(lk), kv), r(sum(lk), kv)


# query and key lengths, heads, kv heads, whether the keys are split
SHAPES = [([150, 70], [150, 70], 4, 2, False),     # single tiles of 128 rows
          ([1300], [1300], 16, 16, False),         # pairs of tiles
          ([130], [1500], 2, 2, True),             # pairs, split
          ([3, 2], [100, 77], 4, 2, False),        # the 16-row kernel
          ([1], [1500], 8, 2, True),               # the same, split: a token over a cache
          ([40], [20], 4, 2, False)]               # the first rows see no key


def _is_split(q, k, heads, kv, seqs):
    p = P.prism_packed_params(seqs=seqs, heads=heads, kv_heads=kv, head_dim=q.shape[-1], q_rows=q.shape[0], k_rows=k.shape[0], causal=1)
    return P.prism_packed_workspace_size(p, P.PRISM_WS_PACKED_FWD) > 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lq,lk,heads,kv,split", SHAPES)
def test_a_query_that_is_not_a_number(lq, lk, heads, kv, split, dim):
    q, k, v = _inputs(lq, lk, heads, kv, dim)
    qo, ko = _ints(ref.offsets(lq)), _ints(ref.offsets(lk))
    assert _is_split(q, k, heads, kv, len(lq)) == split
    att = PackedAttention(heads, kv, dim)
    clean, clean_lse = att.forward(q, k, v, qo, ko), att.lse
    seen = torch.isfinite(clean_lse)
    row, head = q.shape[0] - 1, heads - 1
    q[row, head, 3] = NAN
    o = att.forward(q, k, v, qo, ko)
    dq, dk, dv = att.backward(torch.ones_like(q))
    P.prism_device_status()
    assert seen[head, row]
    assert torch.isnan(o[row, head]).all() and torch.isnan(att.lse[head, row])
    others = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    others[row, head] = False
    assert torch.equal(o[others], clean[others]) and torch.equal(att.lse.T[others], clean_lse.T[others])
    assert (o[~seen.T & others] == 0).all()
    # its gradient, and those of the keys that it sees: all of its sequence's last head, and nothing else
    assert torch.isnan(dq[row, head]).all() and torch.isfinite(dq[others].float()).all()
    last = sum(lk[:-1])
    for g in (dk, dv):
        assert torch.isnan(g[last:, kv - 1]).all()
        assert torch.isfinite(g[:last].float()).all() and torch.isfinite(g[last:, :kv - 1].float()).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lq,lk,heads,kv,split", SHAPES)
def test_a_key_that_is_not_a_number(lq, lk, heads, kv, split, dim):
    """The first key of the last sequence, which every row of it sees that sees any."""
    q, k, v = _inputs(lq, lk, heads, kv, dim)
    qo, ko = _ints(ref.offsets(lq)), _ints(ref.offsets(lk))
    att = PackedAttention(heads, kv, dim, training=False)
    clean, clean_lse = att.forward(q, k, v, qo, ko), att.lse
    k[sum(lk[:-1]), kv - 1, 5] = NAN
    o = att.forward(q, k, v, qo, ko)
    P.prism_device_status()
    hit = torch.isfinite(clean_lse.T).clone()
    hit[:sum(lq[:-1])] = False
    hit[:, :heads - heads // kv] = False
    assert hit.any()
    assert torch.isnan(o[hit]).all() and torch.isnan(att.lse.T[hit]).all()
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(att.lse.T[~hit], clean_lse.T[~hit])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lq,lk,heads,kv,split", SHAPES)
def test_a_value_that_is_not_a_number(lq, lk, heads, kv, split, dim):
    """One element of a value: that column of the rows that see it; the scores do not know of it."""
    q, k, v = _inputs(lq, lk, heads, kv, dim)
    qo, ko = _ints(ref.offsets(lq)), _ints(ref.offsets(lk))
    att = PackedAttention(heads, kv, dim, causal=False, training=False)
    clean, clean_lse = att.forward(q, k, v, qo, ko), att.lse
    v[-1, kv - 1, 5] = NAN
    o = att.forward(q, k, v, qo, ko)
    P.prism_device_status()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[sum(lq[:-1]):, heads - heads // kv:, 5] = True
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit]) and torch.equal(att.lse, clean_lse)
