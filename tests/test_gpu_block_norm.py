"""The norms around a block against the 64-bit reference: a result rounded to bf16 is off by at most U of its
value, statistics and sums in 32 bits by a few 2^-20 of the magnitudes that they sum (values here are O(1))."""

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.packed import BlockNorm, PackedAttention
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SLACK = 2.0 ** -17


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _tol(want, dtype, gain=1.0, mag=0.0):
    return (ref.U * np.abs(want) if dtype == torch.bfloat16 else 0.0) + SLACK * (gain * (1.0 + np.abs(want)) + mag)


def _within(got, want, tol, what):
    over = np.abs(_f64(got).reshape(want.shape) - want) - tol
    assert np.isfinite(_f64(got)).all(), what
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over at {int((over > 0).sum())} of {over.size} places"


def _inputs(n, c, b, stream, branch, param, mods, seed=0, rows=None):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, t, gain=1.0, mean=0.0: (torch.randn(*s, generator=gen) * gain + mean).to(TYPES[t]).cuda()
    a = dict(x=r(n, c, t=stream, mean=0.3), y=r(n, c, t=branch, gain=0.8, mean=-0.1), post_weight=r(c, t=param, gain=0.2, mean=1.0),
             weight=r(c, t=param, gain=0.2, mean=1.0), dh=r(n, c, t=branch), dx_out=r(n, c, t=stream))
    for m in ("gate", "scale", "shift"):
        a[m] = None if mods == "none" else r(c, t=param, gain=0.4) if mods == "shared" else r(b, c, t=param, gain=0.4)
    return a


NAMES = ("post_weight", "gate", "weight", "scale", "shift")


def _reference(a, off, post, pre, alpha, eps=1e-6, grads=True, kept=None, y=True):
    two = lambda t: None if t is None else t if t.ndim == 2 else t[None]
    p = {n: _f64(a.get(n)) for n in NAMES}
    for n in ("gate", "scale", "shift"):
        p[n] = two(p[n])
    return ref.block_norm(_f64(a["x"]), _f64(a["y"]) if y else None, off, post, pre, eps, alpha, **p,
                          dh=_f64(a["dh"]) if grads else None, dx_out=_f64(a["dx_out"]) if grads else None, kept=kept)


def _check_grads(g, a, want, alpha, what):
    _within(g["dx"], want["dx"], _tol(want["dx"], a["x"].dtype, 8.0), what + " dx")
    if g["dy"] is not None:
        _within(g["dy"], want["dy"], _tol(want["dy"], a["y"].dtype, 16.0), what + " dy")
    for n in NAMES:
        if a.get(n) is None or g["d" + n] is None:
            continue
        w = want["d" + n].reshape(g["d" + n].shape)
        _within(g["d" + n], w, _tol(w, a[n].dtype, 4.0, 4.0 * want["abs"]["d" + n].reshape(w.shape)), what + " d" + n)


COMBOS = [("none", "rms"), ("none", "layer"), ("rms", "rms"), ("layer", "layer"), ("rms", "layer"), ("layer", "rms")]


@pytest.mark.parametrize("post,pre", COMBOS)
@pytest.mark.parametrize("stream,branch,param,mods", [("bf16", "bf16", "bf16", "per"), ("f32", "bf16", "f32", "shared"),
                                                      ("bf16", "f32", "f32", "none"), ("f32", "f32", "bf16", "per")])
def test_forward_and_backward(post, pre, stream, branch, param, mods):
    for lens, c in (([37, 0, 1, 130], 256), ([5, 9], 712), ([3], 4104)):
        off = ref.offsets(lens)
        a = _inputs(off[-1], c, len(lens), stream, branch, param, mods)
        norm = BlockNorm(c, post=post, pre=pre, alpha=0.7)
        yn = torch.empty(off[-1], device="cuda")
        x_out, h = norm.forward(a["x"], a["y"], offsets=_ints(off), y_norms=yn, **{n: a[n] for n in NAMES})
        assert x_out.dtype == a["x"].dtype and h.dtype == a["y"].dtype
        g = norm.backward(a["dh"], a["dx_out"])
        P.prism_device_status()
        want = _reference(a, off, post, pre, 0.7, kept=_f64(x_out))
        what = f"{post} {pre} {lens} {c}"
        _within(x_out, want["x_out"], _tol(want["x_out"], x_out.dtype, 4.0), what + " x_out")
        _within(h, want["h"], _tol(want["h"], h.dtype, 8.0), what + " h")
        _within(yn, want["y_norms"], SLACK * want["y_norms"], what + " y_norms")
        _check_grads(g, a, want, 0.7, what)


@pytest.mark.parametrize("c", [8, 16, 248, 256, 264, 1536, 2040, 2056, 4096, 4104, 5120, 8184, 8192])
def test_widths(c):
    """Narrow rows share a CTA, wide ones take several warps or two vectors a thread; ragged last warps."""
    off = ref.offsets([1, 11, 6])
    a = _inputs(18, c, 3, "bf16", "bf16", "f32", "per", seed=c)
    norm = BlockNorm(c, post="rms", pre="layer")
    x_out, h = norm.forward(a["x"], a["y"], offsets=_ints(off), **{n: a[n] for n in NAMES})
    g = norm.backward(a["dh"], a["dx_out"])
    P.prism_device_status()
    want = _reference(a, off, "rms", "layer", 1.0, kept=_f64(x_out))
    _within(x_out, want["x_out"], _tol(want["x_out"], x_out.dtype, 4.0), "x_out")
    _within(h, want["h"], _tol(want["h"], h.dtype, 8.0), "h")
    _check_grads(g, a, want, 1.0, str(c))


@pytest.mark.parametrize("rows", [1, 2, 7, 4099, 20000])
def test_row_counts(rows):
    a = _inputs(rows, 128, 1, "f32", "bf16", "f32", "per", seed=rows)
    norm = BlockNorm(128, post="none", pre="rms")
    x_out, h = norm.forward(a["x"], a["y"], **{n: a[n] for n in NAMES})
    g = norm.backward(a["dh"], a["dx_out"])
    off = ref.offsets([rows])
    want = _reference(a, off, "none", "rms", 1.0, kept=_f64(x_out))
    _within(h, want["h"], _tol(want["h"], h.dtype, 8.0), "h")
    _check_grads(g, a, want, 1.0, str(rows))
    P.prism_device_status()


def test_norm_before_a_block_alone():
    """Without y: h from x, dx without the residual's gradient or with it."""
    off = ref.offsets([20, 30])
    a = _inputs(50, 320, 2, "bf16", "bf16", "bf16", "per")
    norm = BlockNorm(320, post="layer", pre="layer", alpha=0.5)      # alpha and post belong to y: not used
    x_out, h = norm.forward(a["x"], offsets=_ints(off), weight=a["weight"], scale=a["scale"], shift=a["shift"])
    assert x_out is a["x"]
    a.update(gate=None, post_weight=None)
    for with_res in (True, False):
        g = norm.backward(a["dh"], a["dx_out"] if with_res else None)
        b = dict(a) if with_res else dict(a, dx_out=torch.zeros_like(a["dx_out"]))
        want = _reference(b, off, "layer", "layer", 0.5, y=False)
        _within(h, want["h"], _tol(want["h"], h.dtype, 8.0), "h")
        assert g["dy"] is None and g["dgate"] is None
        _check_grads(g, a, want, 1.0, "pre")
    h32 = norm.forward(a["x"], offsets=_ints(off), h_dtype=torch.float32)[1]
    assert h32.dtype == torch.float32
    P.prism_device_status()


def test_rows_of_zeros_and_one_value():
    """A row without variance has nothing but eps to divide by; both norms stay finite."""
    x = torch.zeros(6, 64, device="cuda")
    x[1], x[2] = 3.0, 1e-4
    y = torch.zeros(6, 64, device="cuda")
    for pre in ("rms", "layer"):
        norm = BlockNorm(64, post="layer", pre=pre)
        x_out, h = norm.forward(x, y)
        g = norm.backward(torch.ones_like(y), torch.ones_like(x))
        want = ref.block_norm(_f64(x), _f64(y), ref.offsets([6]), "layer", pre, 1e-6, 1.0, dh=np.ones((6, 64)),
                              dx_out=np.ones((6, 64)))
        # dx sums terms of 1 / sqrt(eps) = 1e3 that cancel: their rounding counts
        for n, t, tol in (("h", h, 1e-4), ("dx", g["dx"], 1e3 * 2.0 ** -14), ("dy", g["dy"], 1e6 * 2.0 ** -14)):
            _within(t, want[n], tol + 1e-4 * np.abs(want[n]), n)


def test_strided_tensors_and_a_modulation_tensor():
    """x, y, h in slices of wider rows; gate, scale and shift as slices of one [sequences, 6, channels] tensor."""
    c, b, n = 512, 3, 90
    off = ref.offsets([30, 0, 60])
    a = _inputs(n, c, b, "bf16", "bf16", "f32", "per")
    mod = torch.randn(b, 6, c, device="cuda") * 0.3
    a.update(scale=mod[:, 1], shift=mod[:, 0], gate=mod[:, 2])
    wide = lambda t: torch.cat([t, torch.full_like(t, 9.0)], 1)[:, :c]
    for m in ("x", "y", "dh", "dx_out"):
        a[m] = wide(a[m])
    outs = {m: torch.full((n, c + 64), 9.0, dtype=torch.bfloat16, device="cuda") for m in ("x_out", "h", "dx", "dy")}
    norm = BlockNorm(c, post="rms", pre="layer", alpha=1.5)
    x_out, h = norm.forward(a["x"], a["y"], offsets=_ints(off), x_out=outs["x_out"][:, :c], h=outs["h"][:, :c],
                            **{m: a[m] for m in NAMES})
    g = norm.backward(a["dh"], a["dx_out"], outs["dx"][:, :c], outs["dy"][:, :c])
    P.prism_device_status()
    want = _reference(a, off, "rms", "layer", 1.5, kept=_f64(x_out))
    _within(x_out, want["x_out"], _tol(want["x_out"], x_out.dtype, 4.0), "x_out")
    _within(h, want["h"], _tol(want["h"], h.dtype, 8.0), "h")
    _check_grads(g, a, want, 1.5, "strided")
    assert all((t[:, c:] == 9.0).all() for t in outs.values())


@pytest.mark.parametrize("c", [256, 1536, 2056, 4104, 8192])
def test_in_place(c):
    """x_out over x, h over y, dx over dx_out, dy over dh: the same bits as in tensors of their own."""
    a = _inputs(1200, c, 1, "bf16", "bf16", "f32", "shared", seed=c)
    kw = {n: a[n] for n in NAMES}
    norm = BlockNorm(c, post="rms", pre="layer", alpha=0.9)
    x_out, h = norm.forward(a["x"], a["y"], **kw)
    g = norm.backward(a["dh"], a["dx_out"])
    x = a["x"].clone()
    over, h2 = norm.forward(x, a["y"], x_out=x, **kw)
    assert over is x and torch.equal(x, x_out) and torch.equal(h2, h)
    dh, dxo = a["dh"].clone(), a["dx_out"].clone()
    g2 = norm.backward(dh, dxo, dx=dxo, dy=dh)
    assert g2["dx"] is dxo and g2["dy"] is dh
    for n in g:
        assert torch.equal(g2[n], g[n]), n
    x, y = a["x"].clone(), a["y"].clone()
    BlockNorm(c, post="rms", pre="layer", alpha=0.9, training=False).forward(x, y, x_out=x, h=y, **kw)
    P.prism_device_status()
    assert torch.equal(x, x_out) and torch.equal(y, h)


def test_refused_places():
    norm = BlockNorm(64)
    x, y = (torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for args, kw in (((x, y), dict(h=y)), ((x,), dict(x_out=y)), ((x, y), dict(x_out=x, h=x))):
        with pytest.raises(P.PrismError) as e:
            norm.forward(*args, **kw)
        assert e.value.code == P.PRISM_EINVAL


def test_rows_outside_the_sequences_stay_as_they_were():
    off = np.array([4, 10, 10, 25], np.int32)
    a = _inputs(40, 96, 3, "bf16", "bf16", "bf16", "per")
    for m in ("x", "y", "dh", "dx_out"):
        a[m][:4], a[m][25:] = float("nan"), float("nan")
    norm = BlockNorm(96, post="rms", pre="rms")
    outs = [torch.full_like(a["x"], 5.0) for _ in range(4)]
    yn = torch.full((40,), 5.0, device="cuda")
    norm.forward(a["x"], a["y"], offsets=_ints(off), x_out=outs[0], h=outs[1], y_norms=yn, **{m: a[m] for m in NAMES})
    g = norm.backward(a["dh"], a["dx_out"], outs[2], outs[3])
    P.prism_device_status()
    for t in outs + [yn]:
        assert (t[:4] == 5.0).all() and (t[25:] == 5.0).all() and torch.isfinite(t[4:25].float()).all()
    clean = {m: None if t is None else torch.nan_to_num(t) for m, t in a.items()}
    kept = _f64(torch.nan_to_num(outs[0]))
    want = _reference(clean, off, "rms", "rms", 1.0, kept=kept)
    for m in NAMES:
        w = want["d" + m].reshape(g["d" + m].shape)
        _within(g["d" + m], w, _tol(w, torch.bfloat16, 4.0, 4.0 * want["abs"]["d" + m].reshape(w.shape)), m)


def test_offsets_out_of_range_are_latched_and_harmless():
    a = _inputs(30, 64, 3, "bf16", "bf16", "f32", "none")
    for bad in ([0, 10, 20, 31], [0, 20, 10, 30], [-2, 10, 20, 30], [30, 20, 10, 0], [0, 10, 20, 1 << 30]):
        norm = BlockNorm(64)
        norm.forward(a["x"], a["y"], offsets=_ints(bad), weight=a["weight"])
        norm.backward(a["dh"], a["dx_out"])
        with pytest.raises(P.PrismError) as e:
            P.prism_device_status()
        assert e.value.code == P.PRISM_EBOUNDS
    P.prism_device_status()


def test_refusals_on_the_device():
    norm = BlockNorm(64)
    x = torch.zeros(6, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for args, kw in (((x[:, :32],), {}), ((x, x[:3]), {}), ((x,), dict(weight=w.cpu())), ((x,), dict(weight=w[:32])),
                     ((x,), dict(weight=w, scale=w.bfloat16())), ((x,), dict(scale=w.expand(3, 64), offsets=_ints([0, 2, 4, 6]))),
                     ((x,), dict(scale=torch.zeros(2, 64, device="cuda"), offsets=_ints([0, 2, 4, 6]))),
                     ((x,), dict(offsets=_ints([0, 6]).long())), ((x.view(2, 3, 64),), dict(offsets=_ints([0, 6]))),
                     ((x,), dict(scale=torch.zeros(4, 64, device="cuda"))), ((x, x), dict(y_norms=torch.zeros(5, device="cuda")))):
        with pytest.raises(P.PrismError) as e:
            norm.forward(*args, **kw)
        assert e.value.code == P.PRISM_EINVAL, (args, kw)
    with pytest.raises(TypeError):
        norm.forward(x.half())
    norm.forward(x, x)
    with pytest.raises(TypeError):
        norm.backward(x.bfloat16())
    with pytest.raises(P.PrismError):
        norm.backward(x[:3])


def test_repeatable_on_streams_and_in_graphs():
    off = _ints(ref.offsets([700, 13, 2000]))
    sets = [_inputs(2713, 384, 3, "bf16", "bf16", "f32", "per", seed=i) for i in range(2)]

    def step(a):
        norm = BlockNorm(384, post="layer", pre="rms")
        x_out, h = norm.forward(a["x"], a["y"], offsets=off, **{n: a[n] for n in NAMES})
        return [x_out, h] + list(norm.backward(a["dh"], a["dx_out"]).values())

    want = [step(a) for a in sets]
    same = lambda p, q: all(torch.equal(s, t) for s, t in zip(p, q))
    assert all(same(step(a), w) for a, w in zip(sets, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(sets[i])
    torch.cuda.synchronize()
    assert all(same(p, q) for p, q in zip(got, want))
    graphs, outs = [], []
    bufs = [{n: None if t is None else t.clone() for n, t in a.items()} for a in sets]
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(b))
        graphs.append(g)
    for i, j in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for n, t in bufs[i].items():
            if t is not None:
                t.copy_(sets[j][n])
        graphs[i].replay()
        assert same(outs[i], want[j])
    P.prism_device_status()
