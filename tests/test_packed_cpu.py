"""Packed-sequence operators without a GPU: the references against finite differences, and every refusal
(bad sizes, strides, pointers and types answer before any CUDA call)."""

import ctypes

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import build, packed, prism as P
from tests import packed_reference as ref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return P.lib()


def _pp(**kw):
    base = dict(seqs=2, heads=4, kv_heads=2, head_dim=128, q_rows=10, k_rows=12, causal=1, scale=0.0)
    base.update({k: v for k, v in kw.items() if not k.endswith("stride")})
    p = P.prism_packed_params(**base)
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(p, k)[:] = v
    return p


def _np(**kw):
    base = dict(rows=10, channels=64, seqs=2, stream_dtype=0, branch_dtype=0, param_dtype=1, post_norm=1, pre_norm=2,
                eps=1e-6, alpha=1.0)
    base.update(kw)
    return P.prism_norm_params(**base)


FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


@pytest.mark.parametrize("causal", [False, True])
def test_attention_reference_gradients_against_differences(causal):
    rng = np.random.default_rng(0)
    qo, ko = ref.offsets([3, 0, 5]), ref.offsets([4, 2, 3])
    q, k, v = rng.normal(size=(8, 4, 6)), rng.normal(size=(9, 2, 6)), rng.normal(size=(9, 2, 6))
    do = rng.normal(size=q.shape)
    out, _, _ = ref.attention(q, k, v, qo, ko, causal, 0.4, dout=do)
    loss = lambda q, k, v: float((ref.attention(q, k, v, qo, ko, causal, 0.4)[0]["o"] * do).sum())
    eps = 1e-5
    for i, n in enumerate(("dq", "dk", "dv")):
        args = [q, k, v]
        for _ in range(12):
            at = tuple(rng.integers(s) for s in args[i].shape)
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[i][at] += eps
            lo[i][at] -= eps
            # the central difference is off by eps^2 times the third derivative, and by rounding / eps
            assert abs((loss(*hi) - loss(*lo)) / (2 * eps) - out[n][at]) < 1e-7


@pytest.mark.parametrize("post,pre,shared", [("none", "layer", True), ("rms", "rms", False), ("layer", "layer", False)])
def test_block_norm_reference_gradients_against_differences(post, pre, shared):
    rng = np.random.default_rng(1)
    off, c = ref.offsets([3, 0, 4]), 6
    mods = 1 if shared else 3
    a = dict(x=rng.normal(size=(7, c)), y=rng.normal(size=(7, c)), post_weight=rng.normal(size=c),
             gate=rng.normal(size=(mods, c)), weight=rng.normal(size=c), scale=rng.normal(size=(mods, c)),
             shift=rng.normal(size=(mods, c)))
    dh, dxo = rng.normal(size=(7, c)), rng.normal(size=(7, c))

    def run(d, **kw):
        return ref.block_norm(d["x"], d["y"], off, post, pre, 1e-3, 0.7, *(d[n] for n in list(d)[2:]), **kw)

    g = run(a, dh=dh, dx_out=dxo)
    loss = lambda d: float((run(d)["h"] * dh).sum() + (run(d)["x_out"] * dxo).sum())
    eps = 1e-5
    for n in a:
        for _ in range(6):
            at = tuple(rng.integers(s) for s in a[n].shape)
            hi, lo = ({m: t.copy() for m, t in a.items()} for _ in range(2))
            hi[n][at] += eps
            lo[n][at] -= eps
            assert abs((loss(hi) - loss(lo)) / (2 * eps) - g["d" + n][at]) < 1e-6, n


@pytest.mark.parametrize("bad,what", [
    (dict(seqs=0), "seqs"), (dict(heads=3), "multiple"), (dict(kv_heads=0), "multiple"), (dict(head_dim=96), "head_dim"),
    (dict(heads=258, kv_heads=2), "128"), (dict(q_rows=-1), "row counts"), (dict(k_rows=2**31), "row counts"),
    (dict(q_rows=2**30), "2\\^31"), (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale")])
def test_packed_params_refused(lib, bad, what):
    for kind in (P.PRISM_WS_PACKED_FWD, P.PRISM_WS_PACKED_BWD):
        with pytest.raises(P.PrismError, match=what) as e:
            P.prism_packed_workspace_size(_pp(**bad), kind)
        assert e.value.code == P.PRISM_EINVAL
    assert lib.prism_packed_attn_fwd(ctypes.byref(_pp(**bad)), *[FAKE] * 6, FAKE, FAKE, FAKE, FAKE, 0, None) == P.PRISM_EINVAL


@pytest.mark.parametrize("bad,what", [
    (dict(q_stride=(512, 12)), "strides"), (dict(k_stride=(-256, 128)), "strides"), (dict(v_stride=(0, 128)), "strides"),
    (dict(o_stride=(256, 128)), "overlap"), (dict(o_stride=(512, 64)), "overlap")])
def test_packed_strides_refused(lib, bad, what):
    rc = lib.prism_packed_attn_fwd(ctypes.byref(_pp(**bad)), *[FAKE] * 6, FAKE, FAKE, FAKE, FAKE, 1 << 40, None)
    assert rc == P.PRISM_EINVAL and what.encode() in lib.prism_last_error()
    if "o_stride" in bad:
        bad = {"dq_stride": bad["o_stride"]}
        rc = lib.prism_packed_attn_bwd(ctypes.byref(_pp(**bad)), *[FAKE] * 13, FAKE, 1 << 40, None)
        assert rc == P.PRISM_EINVAL and what.encode() in lib.prism_last_error()


def test_packed_pointers_refused(lib):
    p = _pp()
    ok = [FAKE] * 10
    for i in (0, 1, 2, 6, 8):       # q, k, v, o, lse
        args = list(ok)
        args[i] = None
        assert lib.prism_packed_attn_fwd(ctypes.byref(p), *args, 1 << 40, None) == P.PRISM_EINVAL
        assert b"NULL" in lib.prism_last_error()
    for i in (0, 1, 2, 6, 7):
        args = list(ok)
        args[i] = ODD
        assert lib.prism_packed_attn_fwd(ctypes.byref(p), *args, 1 << 40, None) == P.PRISM_EINVAL
        assert b"aligned" in lib.prism_last_error()
    # an even split that does not come out even
    odd = _pp(q_rows=11)
    args = list(ok)
    args[3] = None
    assert lib.prism_packed_attn_fwd(ctypes.byref(odd), *args, 1 << 40, None) == P.PRISM_EINVAL
    assert b"evenly" in lib.prism_last_error()
    # backward: workspace
    need = P.prism_packed_workspace_size(p, P.PRISM_WS_PACKED_BWD)
    assert need > 0
    for ws, n in ((None, need), (FAKE, need - 1), (ODD, need)):
        assert lib.prism_packed_attn_bwd(ctypes.byref(p), *[FAKE] * 13, ws, n, None) == P.PRISM_EINVAL
        assert b"workspace" in lib.prism_last_error()
    with pytest.raises(P.PrismError):
        P.prism_packed_workspace_size(p, 99)
    # nothing to do
    empty = _pp(q_rows=0, k_rows=0)
    assert lib.prism_packed_attn_fwd(ctypes.byref(empty), *[None] * 10, 0, None) == P.PRISM_OK


def test_packed_backward_of_nothing_touches_no_device(lib):
    empty = _pp(q_rows=0, k_rows=0)
    assert lib.prism_packed_attn_bwd(ctypes.byref(empty), *[None] * 14, 0, None) == P.PRISM_OK


def _spread(n, **same):
    """n pointers 1 MB apart; `same`: position -> position whose pointer it takes."""
    a = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(n)]
    for i, j in same.items():
        a[int(i[1:])] = a[j]
    return a


@pytest.mark.parametrize("i,j", [(6, 0), (6, 1), (6, 2), (7, 0), (7, 6), (8, 6)])      # o, o_res, lse on q, k, v, o
def test_packed_forward_outputs_on_other_tensors_refused(lib, i, j):
    assert lib.prism_packed_attn_fwd(ctypes.byref(_pp()), *_spread(10, **{f"_{i}": j}), 1 << 40, None) == P.PRISM_EINVAL
    assert b"take the place" in lib.prism_last_error()


@pytest.mark.parametrize("i,j", [(10, 0), (10, 3), (10, 5), (11, 1), (12, 2), (12, 11), (11, 10)])
def test_packed_backward_outputs_on_other_tensors_refused(lib, i, j):
    # q k v o o_res dout lse q_off k_off k_used dq dk dv workspace
    assert lib.prism_packed_attn_bwd(ctypes.byref(_pp()), *_spread(14, **{f"_{i}": j}), 1 << 40, None) == P.PRISM_EINVAL
    assert b"take the place" in lib.prism_last_error()


def test_norm_outputs_on_other_tensors_refused(lib):
    # x y off post_weight gate weight scale shift x_out h y_norms; stream and branch bf16
    for p, i, j in ((_np(), 9, 8), (_np(x_out_row_stride=128), 8, 0), (_np(h_row_stride=72), 9, 1),
                    (_np(stream_dtype=1), 9, 0), (_np(branch_dtype=1), 8, 1)):
        assert lib.prism_block_norm_fwd(ctypes.byref(p), *_spread(11, **{f"_{i}": j}), None) == P.PRISM_EINVAL
        assert b"an input's place" in lib.prism_last_error()
    # x_out y off post_weight gate weight scale dh dx_out dx dy ...
    for p, i, j in ((_np(), 10, 9), (_np(dx_row_stride=72), 9, 8), (_np(dy_row_stride=72), 10, 7), (_np(stream_dtype=1), 9, 7)):
        assert lib.prism_block_norm_bwd(ctypes.byref(p), *_spread(17, **{f"_{i}": j}), 1 << 40, None) == P.PRISM_EINVAL
        assert b"an input's place" in lib.prism_last_error()


@pytest.mark.parametrize("bad,what", [
    (dict(rows=-1), "rows"), (dict(seqs=0), "seqs"), (dict(channels=12), "channels"), (dict(channels=8200), "channels"),
    (dict(stream_dtype=2), "dtypes"), (dict(branch_dtype=-1), "dtypes"), (dict(param_dtype=5), "dtypes"),
    (dict(post_norm=3), "post_norm"), (dict(pre_norm=0), "pre_norm"), (dict(eps=-1.0), "eps"),
    (dict(alpha=float("nan")), "alpha"), (dict(gate_stride=32), "parameter strides"), (dict(shift_stride=68), "parameter strides"),
    (dict(seqs=70000), "65534")])
def test_norm_params_refused(lib, bad, what):
    with pytest.raises(P.PrismError, match=what) as e:
        P.prism_block_norm_workspace_size(_np(**bad))
    assert e.value.code == P.PRISM_EINVAL
    assert lib.prism_block_norm_fwd(ctypes.byref(_np(**bad)), *[FAKE] * 12) == P.PRISM_EINVAL


def test_norm_pointers_refused(lib):
    p = _np()
    for i, want in ((0, b"NULL"), (8, b"NULL")):     # x, x_out (with y)
        args = [FAKE] * 11 + [None]
        args[i] = None
        assert lib.prism_block_norm_fwd(ctypes.byref(p), *args) == P.PRISM_EINVAL and want in lib.prism_last_error()
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9):
        args = [FAKE] * 11 + [None]
        args[i] = ODD
        assert lib.prism_block_norm_fwd(ctypes.byref(p), *args) == P.PRISM_EINVAL and b"aligned" in lib.prism_last_error()
    args = [FAKE, None] + [FAKE] * 9 + [None]        # y_norms without y
    assert lib.prism_block_norm_fwd(ctypes.byref(p), *args) == P.PRISM_EINVAL and b"y_norms" in lib.prism_last_error()
    assert lib.prism_block_norm_fwd(ctypes.byref(_np(x_row_stride=32)), *[FAKE] * 11, None) == P.PRISM_EINVAL
    assert lib.prism_block_norm_fwd(ctypes.byref(_np(rows=11)), FAKE, FAKE, None, *[FAKE] * 8, None) == P.PRISM_EINVAL
    assert b"evenly" in lib.prism_last_error()
    assert lib.prism_block_norm_fwd(ctypes.byref(_np(rows=0)), *[None] * 12) == P.PRISM_OK
    need = P.prism_block_norm_workspace_size(p)
    for ws, n in ((None, need), (FAKE, need - 1), (ODD, need)):
        assert lib.prism_block_norm_bwd(ctypes.byref(p), *[FAKE] * 16, ws, n, None) == P.PRISM_EINVAL
        assert b"workspace" in lib.prism_last_error()
    args = [FAKE] * 17
    args[7] = args[8] = None                          # neither dh nor dx_out
    assert lib.prism_block_norm_bwd(ctypes.byref(p), *args, need, None) == P.PRISM_EINVAL


def test_python_layer_refuses_host_tensors_and_wrong_use():
    att = packed.PackedAttention(4, 2, 64)
    t = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(P.PrismError, match="CUDA"):
        att.forward(t, t, t)
    with pytest.raises(P.PrismError, match="forward"):
        att.backward(t)
    norm = packed.BlockNorm(64)
    with pytest.raises(P.PrismError, match="CUDA"):
        norm.forward(torch.zeros(3, 64))
    with pytest.raises(P.PrismError, match="forward"):
        norm.backward(torch.zeros(3, 64))
    with pytest.raises(P.PrismError, match="one of"):
        packed.BlockNorm(64, post="batch")


@pytest.mark.parametrize("shape,strides,heads,want", [
    ((5, 4, 64), None, 4, (5, None, 256, 64)), ((5, 4, 64), (768, 64, 1), 4, (5, None, 768, 64)),
    ((2, 5, 4, 64), None, 4, (10, 2, 256, 64)), ((1, 4, 64), (8, 64, 1), 4, (1, None, 256, 64)),
    ((3, 1, 2, 64), (640, 8, 64, 1), 2, (3, 3, 640, 64)), ((4, 2, 64), (64, 256, 1), 2, (4, None, 64, 256))])
def test_strided_views_are_read_as_they_lie(shape, strides, heads, want):
    t = torch.zeros(4096, dtype=torch.bfloat16)
    t = t[: int(np.prod(shape))].view(shape) if strides is None else t.as_strided(shape, strides)
    assert packed._heads_view(t.shape, t.stride(), heads, 64, "t") == want


@pytest.mark.parametrize("shape,strides,heads", [
    ((5, 4, 64), (0, 64, 1), 4), ((5, 4, 64), (256, 0, 1), 4), ((2, 5, 4, 64), (2048, 256, 64, 1), 4),
    ((5, 4, 64), (256, 1, 4), 4)])
def test_unreadable_views_are_refused(shape, strides, heads):
    t = torch.zeros(8192, dtype=torch.bfloat16).as_strided(shape, strides)
    with pytest.raises(P.PrismError):
        packed._heads_view(t.shape, t.stride(), heads, 64, "t")
