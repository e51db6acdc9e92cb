"""Attention over keys in shares: each share's forward alone, the results joined by their LSE, and each share's backward
from the joined O and LSE gives its part of the gradients (the parts of dQ add up to the whole)."""

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _params(q, k, heads, kv):
    return P.prism_packed_params(seqs=1, heads=heads, kv_heads=kv, head_dim=q.shape[-1], q_rows=q.shape[0], k_rows=k.shape[0], causal=0)


def _workspace(p, kind):
    return torch.empty(P.prism_packed_workspace_size(p, kind), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("common", [0.0, 13.0])
@pytest.mark.parametrize("n,shares,heads,kv", [(300, (400, 130), 4, 2), (700, (1000, 900), 2, 2)])
def test_shares_of_the_keys_joined(n, shares, heads, kv, common, dim):
    """Of each part the same three roundings as of the whole (tests/test_gpu_packed_common_parts.py): U of its norm. A
    share's rows of dS do not sum to zero, and its dQ has the keys' common part in earnest, times their sum: with a share
    f of the keys the sum's mean square is f (1 - f) of the row's sum of dS^2, and that of the two roundings in it 2/3 U^2
    f, so relative to it they are 1 / (1 - f) times what they are relative to the whole."""
    gen = torch.Generator().manual_seed(dim + n + int(common))
    r = lambda *s: torch.randn(*s, generator=gen)
    m = sum(shares)
    q, dout = (r(n, heads, dim).to(BF16).cuda() for _ in range(2))
    k = (r(m, kv, dim) + common * r(1, kv, dim)).to(BF16).cuda()
    v = r(m, kv, dim).to(BF16).cuda()
    cuts = np.concatenate([[0], np.cumsum(shares)])
    part = [slice(a, b) for a, b in zip(cuts, cuts[1:])]
    lses, outs = [], []
    for s in part:
        p = _params(q, k[s], heads, kv)
        o, res, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(heads, n, device="cuda")
        P.prism_packed_attn_fwd(p, q, k[s], v[s], None, None, None, o, res, lse, _workspace(p, P.PRISM_WS_PACKED_FWD))
        lses.append(lse)
        outs.append(o.float() + res.float())
    lse = torch.logsumexp(torch.stack(lses), 0)
    whole = sum(torch.exp(a - lse).T[:, :, None] * o for a, o in zip(lses, outs))
    whole = whole.contiguous()
    o = whole.to(BF16)
    res = (whole - o.float()).to(BF16)
    f = lambda t: t.double().cpu().numpy()
    Q, K, V, G = (f(t) for t in (q, k, v, dout))
    g = heads // kv
    want = {s: [np.zeros((n, heads, dim)), np.zeros((m, kv, dim)), np.zeros((m, kv, dim))] for s in range(len(part))}
    for h in range(heads):
        z = Q[:, h] @ K[:, h // g].T * dim ** -0.5
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        dp = G[:, h] @ V[:, h // g].T
        ds = w * (dp - (w * dp).sum(1, keepdims=True))
        for i, s in enumerate(part):
            want[i][0][:, h] = ds[:, s] @ K[s, h // g] * dim ** -0.5
            want[i][1][s, h // g] += ds[:, s].T @ Q[:, h] * dim ** -0.5
            want[i][2][s, h // g] += w[:, s].T @ G[:, h]
    for i, s in enumerate(part):
        p = _params(q, k[s], heads, kv)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k[s]), torch.empty_like(v[s])
        P.prism_packed_attn_bwd(p, q, k[s], v[s], o, res, dout, lse, None, None, None, dq, dk, dv, _workspace(p, P.PRISM_WS_PACKED_BWD))
        P.prism_device_status()
        wide = ref.U * np.sqrt(1 / 3 + 2 / 3 / (1 - shares[i] / m)) if common else ref.U
        for name, got, w, tol in (("dq", dq, want[i][0], wide), ("dk", dk, want[i][1][s], ref.U), ("dv", dv, want[i][2][s], ref.U)):
            err = np.linalg.norm(f(got) - w) / np.linalg.norm(w)
            assert err <= tol, f"share {i} {name}: {err:.2e}"
