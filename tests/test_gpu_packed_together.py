"""The packed operators as a layer uses them: norm -> cross-attention of video tokens to packed audio tokens ->
gate, residual and the next norm, whose pass over y also gives the audio input of the block-sparse layer; its
gradients; the same captured in a graph; and a bounded wait that runs out."""

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.attention import PrismSparseAttention
from dynamic_block_sparse_variance_b200.packed import BlockNorm, PackedAttention
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
T, H, W, HEADS, D = 8, 16, 16, 2, 128
N, C = T * H * W, HEADS * D
AUDIO = 300


def _layer_inputs(seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, gain=1.0: torch.randn(*s, generator=gen) * gain
    return dict(x=r(N, C).cuda(), wq=r(C, C, gain=C ** -0.5).to(BF16).cuda(), audio_kv=r(AUDIO, 2 * HEADS, D).to(BF16).cuda(),
                scale=r(1, C, gain=0.3).cuda(), shift=r(1, C, gain=0.3).cuda(), gate=r(1, C, gain=0.5).cuda(),
                w1=(r(C, gain=0.1) + 1).cuda(), w2=(r(C, gain=0.1) + 1).cuda(), dh=r(N, C).to(BF16).cuda(), dx_out=r(N, C).cuda())


def _layer(a):
    """One block: returns what the next layer takes, the norms of y, and all gradients."""
    before = BlockNorm(C, pre="layer")
    att = PackedAttention(HEADS, HEADS, D, causal=False)
    behind = BlockNorm(C, post="rms", pre="rms")
    _, h = before.forward(a["x"], weight=a["w1"], scale=a["scale"], shift=a["shift"], h_dtype=BF16)
    q = (h @ a["wq"]).view(N, HEADS, D)
    y = att.forward(q, a["audio_kv"][:, :HEADS], a["audio_kv"][:, HEADS:], a["q_off"], a["k_off"])
    norms = torch.empty(N, device="cuda")
    x_out, h2 = behind.forward(a["x"], y.view(N, C), gate=a["gate"], weight=a["w2"], y_norms=norms)
    g2 = behind.backward(a["dh"], a["dx_out"])
    dkv = torch.empty_like(a["audio_kv"])
    dq, _, _ = att.backward(g2["dy"].view(N, HEADS, D), dk=dkv[:, :HEADS], dv=dkv[:, HEADS:])
    dq = dq.view(N, C)
    g1 = before.backward(dq @ a["wq"].T, g2["dx"])
    return dict(x_out=x_out, h2=h2, norms=norms, y=y, dx=g1["dx"], dkv=dkv, dwq=h.T @ dq, dgate=g2["dgate"], dscale=g1["dscale"],
                dshift=g1["dshift"], dw1=g1["dweight"], dw2=g2["dweight"])


def _offsets(a):
    a["q_off"], a["k_off"] = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (N, AUDIO))
    return a


def _exact(a):
    """The layer and its gradients in 64 bits by differentiation, without any rounding in between."""
    names = ("x", "wq", "audio_kv", "scale", "shift", "gate", "w1", "w2")
    leaf = {n: a[n].double().requires_grad_() for n in names}
    centred = leaf["x"] - leaf["x"].mean(1, keepdim=True)
    h = centred / torch.sqrt(centred.square().mean(1, keepdim=True) + 1e-6) * leaf["w1"] * (1 + leaf["scale"]) + leaf["shift"]
    q = (h @ leaf["wq"]).view(N, HEADS, D).transpose(0, 1)
    k, v = (leaf["audio_kv"][:, s].transpose(0, 1) for s in (slice(0, HEADS), slice(HEADS, 2 * HEADS)))
    y = (torch.softmax(q @ k.transpose(1, 2) * D ** -0.5, -1) @ v).transpose(0, 1).reshape(N, C)
    x_out = leaf["x"] + leaf["gate"] * (y / torch.sqrt(y.square().mean(1, keepdim=True) + 1e-6))
    h2 = x_out / torch.sqrt(x_out.square().mean(1, keepdim=True) + 1e-6) * leaf["w2"]
    grads = torch.autograd.grad([h2, x_out], list(leaf.values()), [a["dh"].double(), a["dx_out"].double()])
    g = dict(zip(names, grads))
    return dict(x_out=x_out, h2=h2, y=y.view(N, HEADS, D), norms=y.norm(dim=1), dx=g["x"], dkv=g["audio_kv"], dwq=g["wq"], dgate=g["gate"],
                dscale=g["scale"], dshift=g["shift"], dw1=g["w1"], dw2=g["w2"])


def test_layer_and_its_gradients():
    """Roundings on the longest way (h, q, P, y; dh, dy, dS, dq, dq wq, h again): ten of bf16, each at most U of the
    value; the norms and the softmax pass a relative error on with a factor of at most about 2 here (scores
    of order 1). In the 2-norm: 10 U 2, that is 8 %, as the bound; independent roundings stay far below."""
    a = _offsets(_layer_inputs())
    got, want = _layer(a), {n: t.detach() for n, t in _exact(a).items()}
    P.prism_device_status()
    for n, w in want.items():
        g = got[n].double()
        err = float((g - w).norm() / w.norm())
        assert err <= 20 * ref.U, f"{n}: {err:.3e}"


def test_norms_of_y_are_the_sparse_layers_audio_input():
    """The pass behind the cross-attention gives what prism_audio_norms would compute in a pass of its own (the sums
    differ in their order: C terms of 2^-24), and the block-sparse layer runs on it."""
    a = _offsets(_layer_inputs(1))
    out = _layer(a)
    alone = torch.empty(N, device="cuda")
    P.prism_audio_norms(out["y"].view(N, C), alone)
    assert (out["norms"] - alone).abs().max() <= C * 2.0 ** -24 * alone.max()
    gen = torch.Generator().manual_seed(2)
    qkv = [torch.randn(N, HEADS, D, generator=gen).to(BF16).cuda() for _ in range(3)]
    runs = []
    for audio in (out["norms"], alone):
        sparse = PrismSparseAttention(T, H, W, HEADS, D, 2, 0.9)
        runs.append((sparse.forward(*qkv, audio=audio), sparse.rho.clone()))
    P.prism_device_status()
    assert torch.isfinite(runs[0][0].float()).all()
    assert (runs[0][1] - runs[1][1]).abs().max() <= 1e-5      # densities of the same zones


def test_layer_in_a_graph_beside_eager_calls():
    """Captured once, replayed on new inputs, with eager calls of the same objects' inputs in between."""
    a, b = (_offsets(_layer_inputs(s)) for s in (3, 4))
    want = [_layer(t) for t in (a, b)]
    torch.cuda.synchronize()
    buf = {n: t.clone() for n, t in a.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _layer(buf)
    for src, w in ((b, want[1]), (a, want[0]), (b, want[1])):
        for n, t in src.items():
            buf[n].copy_(t)
        g.replay()
        eager = _layer(src)
        for n in w:
            assert torch.equal(out[n], w[n]) and torch.equal(eager[n], w[n]), n
    P.prism_device_status()


@pytest.mark.parametrize("dim,rows", [(128, 600), (64, 600), (128, 300)])
def test_a_wait_that_runs_out_is_reported(dim, rows):
    """The test hook withholds the first P (forward) or P and dS (backward): the waits run out within their limit,
    PRISM_ETIMEOUT is latched, and the next calls give the same results as before, bit for bit."""
    gen = torch.Generator().manual_seed(6)
    q, k, v, dout = (torch.randn(rows, h, dim, generator=gen).to(BF16).cuda() for h in (4, 2, 2, 4))
    att = PackedAttention(4, 2, dim)
    want = (att.forward(q, k, v),) + att.backward(dout)
    P.prism_device_status()
    try:
        P.prism_set_option(P.PRISM_OPT_WAIT_LIMIT, 20000)
        P.prism_set_option(P.PRISM_OPT_DEBUG_STALL, 1)
        stalled = PackedAttention(4, 2, dim)
        stalled.forward(q, k, v)
        with pytest.raises(P.PrismError) as e:
            P.prism_device_status()
        assert e.value.code == P.PRISM_ETIMEOUT
        att.backward(dout)
        with pytest.raises(P.PrismError) as e:
            P.prism_device_status()
        assert e.value.code == P.PRISM_ETIMEOUT
    finally:
        P.prism_set_option(P.PRISM_OPT_DEBUG_STALL, 0)
        P.prism_set_option(P.PRISM_OPT_WAIT_LIMIT, 0)
    again = (att.forward(q, k, v),) + att.backward(dout)
    P.prism_device_status()
    assert all(torch.equal(x, y) for x, y in zip(again, want))


def test_long_walks_are_cut_the_same_way_every_time():
    """Many query heads on few kv heads: the backward's walks over the queries are cut into shares. Against the
    reference, with keys not in use, rows outside, and bit-equal from run to run."""
    gen = torch.Generator().manual_seed(9)
    heads, kv, d = 14, 1, 128
    qo, ko, used = np.array([2, 2, 500, 690], np.int32), np.array([1, 60, 560, 900], np.int32), np.array([0, 411, 340], np.int32)
    q, dout = (torch.randn(700, heads, d, generator=gen).to(BF16).cuda() for _ in range(2))
    k, v = (torch.randn(910, kv, d, generator=gen).to(BF16).cuda() for _ in range(2))
    ints = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
    for t in (k, v):
        t[:1], t[900:] = float("nan"), float("nan")
        for b in range(3):
            t[ko[b] + used[b]:ko[b + 1]] = float("nan")
    for causal in (True, False):
        att = PackedAttention(heads, kv, d, causal=causal)
        runs = []
        for _ in range(2):
            dk, dv = (torch.full_like(k, 7.0) for _ in range(2))
            att.forward(q, k, v, ints(qo), ints(ko), k_used=ints(used))
            runs.append(att.backward(dout, dk=dk, dv=dv))
        P.prism_device_status()
        assert all(torch.equal(x[2:690], y[2:690]) if x.shape[0] == 700 else torch.equal(x, y) for x, y in zip(*runs))
        f = lambda t: torch.nan_to_num(t).double().cpu().numpy()
        want, bound, _ = ref.attention(f(q), f(k), f(v), qo, ko, causal, d ** -0.5, used, f(dout))
        for n, g, lo, hi in (("dq", runs[0][0], 2, 690), ("dk", runs[0][1], 1, 900), ("dv", runs[0][2], 1, 900)):
            g = g.double().cpu().numpy()
            assert (np.abs(g[lo:hi] - want[n][lo:hi]) <= bound[n][lo:hi]).all(), (n, causal)
            if n != "dq":
                assert (g[:lo] == 7.0).all() and (g[hi:] == 7.0).all()


def test_backward_on_another_stream_keeps_what_the_forward_left():
    """The next forward, on the first stream, lets go of what a late backward on another stream still reads; what
    is allocated then must not be that memory."""
    gen = torch.Generator().manual_seed(9)
    q, k, v, dout = (torch.randn(900, 4, 128, generator=gen).to(BF16).cuda() for _ in range(4))
    x, y, dh = (torch.randn(900, 512, generator=gen).to(BF16).cuda() for _ in range(3))
    att, norm = PackedAttention(4, 4, 128), BlockNorm(512, post="rms")
    att.forward(q, k, v)
    norm.forward(x, y)
    want = [*att.backward(dout), *(norm.backward(dh)[n] for n in ("dx", "dy"))]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(a):
            att.forward(q, k, v)
            norm.forward(x, y)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            torch.cuda._sleep(20_000_000)           # some 10 ms: the backward starts after all that follows
            got = [*att.backward(dout), *(norm.backward(dh)[n] for n in ("dx", "dy"))]
        with torch.cuda.stream(a):
            att.forward(q, k, v)
            norm.forward(x, y)
            for shape, dtype in (((900, 4, 128), BF16), ((4, 900), torch.float32), ((900, 512), BF16)) * 4:
                torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        torch.cuda.synchronize()
        P.prism_device_status()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
