"""Dense attention over packed sequences against the 64-bit reference, elementwise within the bounds that
its roundings allow (tests/packed_reference.py), at the sizes and masks where such kernels go wrong."""

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.packed import PackedAttention
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN = float("nan")


def _f64(t):
    return t.detach().double().cpu().numpy()


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _randn(gen, *shape, gain=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * gain + mean).to(BF16).cuda()


def _within(got, want, bound, what):
    got = _f64(got)
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin), f"{what}: non-finite values in other places"
    assert np.array_equal(got[~fin], want[~fin]), what
    over = np.abs(got[fin] - want[fin]) - np.broadcast_to(bound, want.shape)[fin]
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over the bound at {int((over > 0).sum())} of {over.size} places"


def _close_on_average(got, want, what, rest=0.0):
    """Independent roundings (operand, D, result) have a mean square of at most U^2 / 3 each; `rest`: what sums
    in 32 bits may add where terms cancel (tests/packed_reference.py)."""
    got = _f64(got)
    fin = np.isfinite(want)
    norm = np.linalg.norm(want[fin])
    assert np.linalg.norm(got[fin] - want[fin]) <= np.sqrt(3 * ref.U ** 2 / 3) * norm + np.linalg.norm(rest) + 1e-30, what


def _check(q, k, v, dout, qo, ko, causal, scale, used, att, o, grads=None, what="", average=False):
    want, bound, *rest = ref.attention(_f64(q), _f64(k), _f64(v), qo, ko, causal, scale or q.shape[-1] ** -0.5, used,
                                       _f64(dout) if grads else None)
    rows = np.zeros(q.shape[0], bool)
    for a, b in zip(qo[:-1], qo[1:]):
        rows[a:b] = True
    _within(o[torch.from_numpy(rows).cuda()], want["o"][rows], bound["o"][rows], what + " o")
    _within(att.lse[:, torch.from_numpy(rows).cuda()], want["lse"][:, rows], bound["lse"][:, rows], what + " lse")
    if grads:
        for n, g in zip(("dq", "dk", "dv"), grads):
            off = qo if n == "dq" else ko
            _within(g[off[0]:off[-1]], want[n][off[0]:off[-1]], bound[n][off[0]:off[-1]], what + " " + n)
            if average:
                _close_on_average(g[off[0]:off[-1]], want[n][off[0]:off[-1]], what + " " + n, rest[0][n])
    if average:
        _close_on_average(o[torch.from_numpy(rows).cuda()], want["o"][rows], what + " o")


# lengths: (queries per sequence, keys per sequence or None for the same)
SHAPES = [
    ("one token", [1], None, 1, 1), ("two tokens", [2], None, 2, 1), ("tile edges", [127, 128, 129], None, 2, 2),
    ("beyond a pair of tiles", [255, 257, 1, 0, 3], None, 4, 2), ("empty ends", [0, 0, 5, 0, 70, 0], None, 3, 1),
    ("grouped by five", [33, 90, 26], None, 5, 1), ("grouped by seven", [41, 200], None, 7, 1),
    ("many heads of one", [19, 64], None, 48, 1), ("cross", [50, 3, 0, 129], [20, 300, 7, 129], 4, 2),
    ("keys only in some", [10, 20, 30], [0, 500, 1], 2, 2), ("long", [1100], None, 2, 1),
    ("short queries, long keys", [1, 3, 17], [700, 1025, 129], 8, 2),
    ("more queries than keys", [200, 130], [3, 64], 2, 1),
]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_forward_and_backward(shape, causal, dim):
    name, lq, lk, heads, kv = shape
    gen = torch.Generator().manual_seed(len(name) + dim)
    qo, ko = ref.offsets(lq), ref.offsets(lq if lk is None else lk)
    q, dout = (_randn(gen, qo[-1], heads, dim, gain=g) for g in (1.5, 1.0))
    k, v = (_randn(gen, ko[-1], kv, dim, gain=g, mean=m) for g, m in ((1.5, 0.0), (1.0, 0.2)))
    att = PackedAttention(heads, kv, dim, causal=causal)
    o = att.forward(q, k, v, _ints(qo), _ints(ko))
    grads = att.backward(dout)
    P.prism_device_status()
    _check(q, k, v, dout, qo, ko, causal, 0.0, None, att, o, grads, name, average=True)


@pytest.mark.parametrize("dim,heads,kv", [(128, 2, 2), (128, 4, 1), (64, 3, 1)])
def test_a_tile_without_keys_beside_one_that_has_some(dim, heads, kv):
    """Causal with more queries than keys, enough keys for pairs of 128-row tiles, and a first seen key in the
    second tile of a pair: the first tile's zeros and its queries, which nobody reads, go to the same memory."""
    gen = torch.Generator().manual_seed(dim + heads)
    group = heads // kv
    blind = (256 + 128 + group) // group            # rows up to 128 .. 256 + a token of the second pair see nothing
    lq, lk = [600 + blind, 520, 640 + blind], [600, 520, 640]
    qo, ko = ref.offsets(lq), ref.offsets(lk)
    q, dout = (_randn(gen, qo[-1], heads, dim) for _ in range(2))
    k, v = (_randn(gen, ko[-1], kv, dim) for _ in range(2))
    att = PackedAttention(heads, kv, dim)
    first = None
    for _ in range(50):
        o = att.forward(q, k, v, _ints(qo), _ints(ko))
        P.prism_device_status()
        for s in (qo[0], qo[2]):
            assert (o[s:s + blind] == 0).all() and torch.isneginf(att.lse[:, s:s + blind]).all()
        first = o if first is None else first
        assert torch.equal(o, first)
    _check(q, k, v, dout, qo, ko, True, 0.0, None, att, o, att.backward(dout), "blind rows", average=True)


@pytest.mark.parametrize("dim,heads,kv", [(128, 4, 2), (64, 6, 2)])
def test_what_lies_outside_the_sequences_reaches_nothing(dim, heads, kv):
    """NaN before, between and behind the sequences' rows and behind k_used; rows outside stay as they were."""
    gen = torch.Generator().manual_seed(3)
    qo, ko = np.array([5, 40, 40, 170], np.int32), np.array([3, 150, 160, 420], np.int32)
    used = np.array([101, 0, 259], np.int32)
    q, dout = (_randn(gen, 200, heads, dim) for _ in range(2))
    k, v = (_randn(gen, 450, kv, dim) for _ in range(2))
    q[:5], q[170:], dout[:5], dout[170:] = NAN, NAN, NAN, NAN
    for t in (k, v):
        t[:3], t[420:] = NAN, NAN
        for b in range(3):
            t[ko[b] + used[b]:ko[b + 1]] = NAN
    for causal in (True, False):
        att = PackedAttention(heads, kv, dim, causal=causal)
        out, dq = (torch.full_like(q, 7.0) for _ in range(2))
        dk, dv = (torch.full_like(k, 7.0) for _ in range(2))
        o = att.forward(q, k, v, _ints(qo), _ints(ko), k_used=_ints(used), out=out)
        assert o is out
        att.backward(dout, dq, dk, dv)
        P.prism_device_status()
        clean = [torch.nan_to_num(t) for t in (q, k, v, dout)]
        _check(*clean, qo, ko, causal, 0.0, used, att, o, (dq, dk, dv), "poisoned")
        for t, lo, hi in ((o, 5, 170), (dq, 5, 170), (dk, 3, 420), (dv, 3, 420)):
            assert (t[:lo] == 7.0).all() and (t[hi:] == 7.0).all()
        for t in (dk, dv):          # rows with room but not in use: zero gradients
            for b in range(3):
                assert (t[ko[b] + used[b]:ko[b + 1]] == 0).all()


def test_masked_scores_that_are_not_finite():
    """Infinite and NaN keys in masked (future) places do not reach the scores; their values are finite."""
    gen = torch.Generator().manual_seed(5)
    q, k, v = (_randn(gen, 200, 2, 128) for _ in range(3))
    k[190:] = float("inf")
    k[195] = NAN
    att = PackedAttention(2, 2, 128, training=False)
    o = att.forward(q, k, v)
    full = att.forward(q[:190].contiguous(), k[:190].contiguous(), v[:190].contiguous())
    assert torch.equal(o[:190], full) and torch.isfinite(o[:190].float()).all()


@pytest.mark.parametrize("gain", [0.0, 30.0])
def test_flat_and_peaked_rows(gain):
    """All scores equal, and scores hundreds apart (probabilities underflow, the maximum moves)."""
    gen = torch.Generator().manual_seed(8)
    q, k = (_randn(gen, 600, 2, 128, gain=gain) for _ in range(2))
    v, dout = (_randn(gen, 600, 2, 128) for _ in range(2))
    att = PackedAttention(2, 2, 128)
    o = att.forward(q, k, v)
    off = ref.offsets([600])
    if gain == 0.0:
        _check(q, k, v, dout, off, off, True, 0.0, None, att, o, att.backward(dout), "flat")
    else:
        # scores near 1e4: their 32-bit error, 2^-23 of sum |q k| (about 6e4 scale) is the bound of log p
        want, bound = ref.attention(_f64(q), _f64(k), _f64(v), off, off, True, 128 ** -0.5)
        z = 128 ** -0.5 * np.abs(_f64(q)).max() * np.abs(_f64(k)).sum(-1).max()
        extra = 2.0 ** -20 * z * np.abs(_f64(v)).max()
        _within(o, want["o"], bound["o"] + extra, "peaked o")
        _within(att.lse, want["lse"], bound["lse"] + 2.0 ** -20 * z, "peaked lse")


def test_strided_views_and_scale():
    """q, k, v as slices of one projection's output, outputs and gradients into slices, a scale of one's own."""
    gen = torch.Generator().manual_seed(11)
    heads, kv, d, n = 6, 2, 64, 300
    qkv = _randn(gen, n, heads + 2 * kv, d)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    dout = _randn(gen, n, heads, 2 * d)[:, :, :d]
    off = ref.offsets([120, 180])
    att = PackedAttention(heads, kv, d, scale=0.3)
    room = torch.zeros(n, heads, 3 * d, dtype=BF16, device="cuda")
    o = att.forward(q, k, v, _ints(off), out=room[:, :, d:2 * d])
    dqkv = torch.zeros_like(qkv)
    grads = att.backward(dout, dqkv[:, :heads], dqkv[:, heads:heads + kv], dqkv[:, heads + kv:])
    P.prism_device_status()
    _check(q, k, v, dout, off, off, True, 0.3, None, att, o, grads, "strided")
    assert (room[:, :, :d] == 0).all() and (room[:, :, 2 * d:] == 0).all()
    heads_first = torch.empty(heads, n, d, dtype=BF16, device="cuda").copy_(q.transpose(0, 1)).transpose(0, 1)
    again = PackedAttention(heads, kv, d, scale=0.3).forward(heads_first, k, v, _ints(off))
    assert torch.equal(again, o)


@pytest.mark.parametrize("dim,heads,kv,seqs,tokens,room", [
    (128, 8, 2, 1, 1, 1), (128, 8, 2, 1, 1, 5000), (64, 8, 1, 3, 1, 777), (128, 32, 8, 5, 1, 1500), (128, 12, 2, 2, 5, 400),
    (64, 4, 4, 40, 1, 129), (128, 40, 1, 2, 1, 3001), (128, 2, 1, 1, 16, 2100)])
def test_tokens_over_caches(dim, heads, kv, seqs, tokens, room):
    gen = torch.Generator().manual_seed(room)
    q = _randn(gen, seqs, tokens, heads, dim, gain=1.3)
    k, v = (_randn(gen, seqs, room, kv, dim, gain=1.3) for _ in range(2))
    used = np.random.default_rng(room).integers(min(tokens, room), room + 1, seqs).astype(np.int32)
    used[-1] = room
    for b in range(seqs):
        k[b, used[b]:], v[b, used[b]:] = NAN, NAN
    att = PackedAttention(heads, kv, dim, training=False)
    o = att.forward(q, k, v, k_used=_ints(used))
    P.prism_device_status()
    assert o.shape == q.shape
    flat = lambda t: torch.nan_to_num(t).flatten(0, 1)
    _check(flat(q), flat(k), flat(v), None, ref.offsets([tokens] * seqs), ref.offsets([room] * seqs), True, 0.0, used,
           att, o.flatten(0, 1), what="cache", average=True)


def test_cache_beyond_32_bit_offsets():
    """Two caches of 9.2 million rows each: the second one's elements lie past 2^31 (and bytes past 2^32)."""
    heads, kv, d, room = 4, 2, 128, 9_200_000
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.empty(2, room, kv, d, dtype=BF16, device="cuda") for _ in range(2))
    used = np.array([3, 300], np.int32)
    small = [_randn(gen, 300, kv, d) for _ in range(2)]
    for big, s in zip((k, v), small):
        big[0, :3], big[1, :300] = s[:3], s
    q = _randn(gen, 2, 1, heads, d)
    att = PackedAttention(heads, kv, d, training=False)
    o = att.forward(q, k, v, k_used=_ints(used))
    P.prism_device_status()
    for b in range(2):
        want, bound = ref.attention(_f64(q[b]), _f64(small[0][:used[b]]), _f64(small[1][:used[b]]), ref.offsets([1]),
                                    ref.offsets([used[b]]), True, d ** -0.5)
        _within(o[b], want["o"], bound["o"], f"cache {b}")
    # and a prompt over the far cache
    q2 = _randn(gen, 2, 130, heads, d)
    used2 = np.array([3, 300], np.int32)
    o2 = att.forward(q2, k, v, k_used=_ints(used2))
    want, bound = ref.attention(_f64(q2[1]), _f64(small[0]), _f64(small[1]), ref.offsets([130]), ref.offsets([300]), True,
                                d ** -0.5)
    P.prism_device_status()
    _within(o2[1], want["o"], bound["o"], "prompt over the far cache")


def test_offsets_out_of_range_are_latched_and_harmless():
    """Offsets that leave the tensors or run backwards, and k_used beyond the room: PRISM_EBOUNDS, the other
    sequences' results, and nothing written elsewhere."""
    gen = torch.Generator().manual_seed(2)
    q, k, v = (_randn(gen, 300, 2, 64) for _ in range(3))
    good = PackedAttention(2, 2, 64, training=False).forward(q, k, v, _ints([0, 100, 200, 300]))
    for qo, ko, used, fine in (([0, 100, 200, 301], [0, 100, 200, 300], None, slice(0, 200)),
                               ([0, 100, 200, 300], [0, 100, 200, 1 << 30], None, slice(0, 200)),
                               ([0, 100, 200, 300], [0, 100, 200, 300], [100, 100, 101], slice(0, 200))):
        for train in (False, True):
            att = PackedAttention(2, 2, 64, training=train)
            out = torch.full_like(q, 5.0)
            att.forward(q, k, v, _ints(qo), _ints(ko), k_used=None if used is None else _ints(used), out=out)
            with pytest.raises(P.PrismError) as e:
                P.prism_device_status()
            assert e.value.code == P.PRISM_EBOUNDS
            assert torch.equal(out[fine], good[fine])
            if train:
                att.backward(out)
                with pytest.raises(P.PrismError) as e:
                    P.prism_device_status()
                assert e.value.code == P.PRISM_EBOUNDS
    for bad in ([0, 200, 100, 300], [-1, 100, 200, 300], [300, 200, 100, 0]):
        att = PackedAttention(2, 2, 64)
        o = att.forward(q, k, v, _ints(bad))
        att.backward(o)
        with pytest.raises(P.PrismError) as e:
            P.prism_device_status()
        assert e.value.code == P.PRISM_EBOUNDS
    P.prism_device_status()


def test_refusals_on_the_device():
    att = PackedAttention(4, 2, 64)
    q, k = torch.zeros(10, 4, 64, dtype=BF16, device="cuda"), torch.zeros(10, 2, 64, dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        att.forward(q.float(), k, k)
    for args, kw in (((q, k, k[:5]), {}), ((q[:, :3], k, k), {}), ((q, k, k, _ints([0, 10]).long()), {}),
                     ((q, k, k, _ints([0, 10]), _ints([0, 5, 10])), {}), ((q, k, k), dict(k_used=_ints([1, 2, 3]))),
                     ((q, k, k), dict(out=q[:5])), ((q, k, k.cpu()), {}), ((q, k, k, torch.tensor([0, 10], dtype=torch.int32)), {}),
                     ((q[:1].expand(10, 4, 64), k, k), {}), ((q, k.expand(10, 2, 64)[:, :1].expand(10, 2, 64), k), {})):
        with pytest.raises(P.PrismError) as e:
            att.forward(*args, **kw)
        assert e.value.code == P.PRISM_EINVAL
    att.forward(q, k, k)
    for args in ((q[:5],), (q.cpu(),), (q, q[:5]), (q, torch.zeros_like(q), k[:, :1].expand(10, 2, 64))):
        with pytest.raises(P.PrismError) as e:
            att.backward(*args)
        assert e.value.code == P.PRISM_EINVAL


def test_outputs_on_other_tensors_refused():
    q = torch.zeros(10, 4, 64, dtype=BF16, device="cuda")
    att = PackedAttention(4, 4, 64)
    for args, kw in (((q, q, q), dict(out=q)), ((torch.zeros_like(q), q, torch.zeros_like(q)), dict(out=q))):
        with pytest.raises(P.PrismError) as e:
            att.forward(*args, **kw)
        assert e.value.code == P.PRISM_EINVAL
    o = att.forward(q, q, q)            # one tensor may be read three times
    g = torch.ones_like(q)
    for args in ((g, g), (g, o), (g, None, q), (g, None, torch.zeros_like(q), o)):
        with pytest.raises(P.PrismError) as e:
            att.backward(*args)
        assert e.value.code == P.PRISM_EINVAL
    d = torch.zeros_like(q)
    with pytest.raises(P.PrismError):
        att.backward(g, None, d, d)
    assert all(torch.isfinite(t.float()).all() for t in att.backward(g))


def test_no_rows():
    q, k = torch.zeros(0, 4, 64, dtype=BF16, device="cuda"), torch.zeros(6, 2, 64, dtype=BF16, device="cuda")
    att = PackedAttention(4, 2, 64)
    for qs, ks, qo, ko in ((q, k, [0, 0], [0, 6]), (q, k[:0], [0, 0], [0, 0]), (q, k[:0], [0], [0])):
        o = att.forward(qs, ks, ks, _ints(qo), _ints(ko))
        dq, dk, dv = att.backward(o)
        assert o.shape == qs.shape and dk.shape == ks.shape and (dk == 0).all() and (dv == 0).all()
    q = torch.ones(7, 4, 64, dtype=BF16, device="cuda")
    o = att.forward(q, k[:0], k[:0], _ints([0, 7]), _ints([0, 0]))
    assert (o == 0).all() and torch.isinf(att.lse).all() and (att.backward(q)[0] == 0).all()
    P.prism_device_status()


@pytest.mark.parametrize("heads,kv,dim", [(100, 1, 64), (128, 1, 128), (65, 1, 128), (256, 2, 64)])
def test_a_tile_per_token(heads, kv, dim):
    """Groups so large that a tile of 128 rows holds one token, whole or cut."""
    gen = torch.Generator().manual_seed(heads)
    qo = ref.offsets([5, 0, 130])
    q, dout = (_randn(gen, qo[-1], heads, dim) for _ in range(2))
    k, v = (_randn(gen, qo[-1], kv, dim) for _ in range(2))
    for causal in (True, False):
        att = PackedAttention(heads, kv, dim, causal=causal)
        o = att.forward(q, k, v, _ints(qo))
        grads = att.backward(dout)
        P.prism_device_status()
        _check(q, k, v, dout, qo, qo, causal, 0.0, None, att, o, grads, f"{heads} heads", average=True)


def test_graph_replayed_over_other_lengths():
    """Offsets and lengths are read on the device: a captured step, and a captured token over growing caches, serve
    what the arrays hold when they are replayed."""
    gen = torch.Generator().manual_seed(31)
    q, k, v, dout = (_randn(gen, 1200, h, 128) for h in (4, 2, 2, 4))
    lens = [[1200, 0, 0], [0, 1, 1199], [400, 500, 300], [100, 0, 900]]
    off = _ints(ref.offsets(lens[2]))
    cache_k, cache_v, tok = _randn(gen, 3, 900, 2, 128), _randn(gen, 3, 900, 2, 128), _randn(gen, 3, 4, 128)
    used = _ints([1, 2, 3])
    att, dec = PackedAttention(4, 2, 128), PackedAttention(4, 2, 128, training=False)
    out, dq = (torch.zeros_like(q) for _ in range(2))
    dk, dv = (torch.zeros_like(k) for _ in range(2))

    def step():
        att.forward(q, k, v, off, out=out)
        att.backward(dout, dq, dk, dv)
        return dec.forward(tok, cache_k, cache_v, k_used=used)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        token = step()
    lse, dec_lse = att.lse, dec.lse
    for n, ls in enumerate(lens):
        qo, have = ref.offsets(ls), np.array([900 - n, 300 * n, 17 + n], np.int32)
        off.copy_(_ints(qo))
        used.copy_(_ints(have))
        g.replay()
        P.prism_device_status()
        att.lse, dec.lse = lse, dec_lse
        _check(q, k, v, dout, qo, qo, True, 0.0, None, att, out, (dq, dk, dv), f"lengths {ls}")
        flat = lambda t: t.reshape(2700, 2, 128)
        _check(tok, flat(cache_k), flat(cache_v), None, np.arange(4), np.arange(4) * 900, True, 0.0, have, dec, token,
               what=f"used {have}")


@pytest.mark.parametrize("dim", [64, 128])
def test_repeatable_on_streams_and_in_graphs(dim):
    """Bit-equal results run to run, on two streams at once, and from two captured graphs that are replayed
    in turn with new inputs in the captured buffers."""
    gen = torch.Generator().manual_seed(21)
    off = _ints(ref.offsets([130, 300, 70]))
    sets = [[_randn(gen, 500, h, dim) for h in (4, 2, 2, 4)] for _ in range(2)]

    def step(q, k, v, dout):
        att = PackedAttention(4, 2, dim)
        o = att.forward(q, k, v, off)
        return (o, att.lse) + att.backward(dout)

    want = [step(*s) for s in sets]
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(same(step(*s), w) for s, w in zip(sets, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(*sets[i])
    torch.cuda.synchronize()
    assert all(same(g, w) for g, w in zip(got, want))
    graphs, bufs, outs = [], [], []
    for i in range(2):
        b = [t.clone() for t in sets[i]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*b))
        graphs.append(g)
        bufs.append(b)
    for i, j in ((0, 0), (1, 1), (0, 1), (1, 0), (0, 0)):
        for dst, src in zip(bufs[i], sets[j]):
            dst.copy_(src)
        graphs[i].replay()
        assert same(outs[i], want[j])
    streams = [torch.cuda.Stream() for _ in range(2)]     # both at once
    for i in range(2):
        for dst, src in zip(bufs[i], sets[i]):
            dst.copy_(src)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(outs, want))
    P.prism_device_status()


def test_gradients_against_differences():
    """The directional derivative of sum(dout o) along random directions, by central differences of the 64-bit
    reference, against the kernel's gradients. Bound: the gradients' own elementwise bounds times |direction|."""
    gen = torch.Generator().manual_seed(4)
    qo = ko = ref.offsets([60, 140])
    t = [_randn(gen, 200, h, 64) for h in (4, 2, 2, 4)]
    att = PackedAttention(4, 2, 64)
    att.forward(*t[:3], _ints(qo))
    grads = att.backward(t[3])
    q, k, v, do = (_f64(x) for x in t)
    _, bound, _ = ref.attention(q, k, v, qo, ko, True, 0.125, dout=do)
    loss = lambda *a: float((ref.attention(*a, qo, ko, True, 0.125)[0]["o"] * do).sum())
    rng = np.random.default_rng(0)
    for i, n in enumerate(("dq", "dk", "dv")):
        d = rng.normal(size=(q, k, v)[i].shape)
        hi, lo = ([x + s * 1e-5 * d if j == i else x for j, x in enumerate((q, k, v))] for s in (1, -1))
        diff = (loss(*hi) - loss(*lo)) / 2e-5
        assert abs(diff - float((_f64(grads[i]) * d).sum())) <= float((bound[n] * np.abs(d)).sum()) + 1e-6 * abs(diff)
