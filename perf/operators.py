"""Measured cases of the packed-sequence operators: dense attention over packed sequences (forward, training
pass, single-token serving) and the norms around a block fused with its gate and residual scale.

``own`` False computes them in their plain form (elementary torch operations in 32 bits, rounded once);
``own`` True makes the calls of ``dynamic_block_sparse_variance_b200.packed``.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------

def _attend(name, mode, heads, kv_heads, dim, causal, seqs, q_rows, k_rows, cut):
    return {"name": name, "op": "attend", "pass": mode, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "causal": causal, "seqs": seqs, "q_rows": q_rows, "k_rows": k_rows, "cut": cut}


def _decode(name, heads, kv_heads, dim, seqs, tokens, room, cut):
    return {"name": name, "op": "decode", "heads": heads, "kv_heads": kv_heads, "dim": dim, "seqs": seqs,
            "tokens": tokens, "room": room, "cut": cut}


def _norm(name, mode, rows, channels, seqs, post, pre, stream, branch, param, mods, cut):
    return {"name": name, "op": "norm", "pass": mode, "rows": rows, "channels": channels, "seqs": seqs, "post": post,
            "pre": pre, "stream": stream, "branch": branch, "param": param, "mods": mods, "cut": cut}


def listed():
    return [
        # a batch of prompts of different lengths packed into one call, grouped heads
        _attend("prompts", "forward", 16, 4, 128, True, 9, 8192, 0, 3),
        # one long prompt
        _attend("long prompt", "forward", 8, 8, 128, True, 1, 16384, 0, 0),
        # video tokens of several samples attending to their conditioning tokens, head_dim 64
        _attend("conditioning", "forward", 12, 12, 64, False, 4, 7680, 1111, 5),
        # a training step over packed samples, grouped heads, causal
        _attend("packed training", "train", 16, 4, 128, True, 7, 6144, 0, 11),
        # a training step of one dense self-attention layer (the layers that stay dense), bidirectional
        _attend("dense training", "train", 8, 8, 128, False, 1, 8192, 0, 0),
        # a short training step with odd lengths, head_dim 64
        _attend("short training", "train", 6, 2, 64, True, 3, 777, 0, 7),
        # one user's next token
        _decode("next token", 8, 2, 128, 1, 1, 1500, 1),
        # next tokens of a batch over caches filled to different lengths
        _decode("batch of tokens", 32, 8, 128, 48, 1, 8192, 2),
        # the block between two layers of one grid of 16 x 48 x 80 tokens, 12 heads of 128
        _norm("grid block", "forward", 61440, 1536, 1, "none", "layer", "bf16", "bf16", "f32", True, 0),
        # the same block for a handful of tokens
        _norm("few rows", "forward", 24, 2048, 3, "rms", "rms", "bf16", "bf16", "bf16", False, 4),
        # a training step through the block, modulated per packed sample
        _norm("block training", "train", 30011, 2048, 5, "rms", "layer", "bf16", "bf16", "bf16", True, 6),
        # a training step with the residual stream kept in 32 bits, wide rows
        _norm("wide training", "train", 9001, 5120, 2, "none", "rms", "f32", "bf16", "f32", False, 8),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "train", "decode", "norm", "norm train"])
    cut = rng.randrange(1, 1 << 20)
    if kind in ("attend", "train"):
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 1, 2, 4, 5, 7])
        heads = heads if heads <= 16 else kv_heads
        top = (16384 if kind == "attend" else 8192) * math.sqrt(min(1.0, 8 / heads) * (1.0 if kind == "attend" else 0.9))
        # gradients of q and k where every row sees one key are zero: a training step has longer sequences
        train = kind == "train"
        q_rows = _log_int(rng, 32 if train else 1, top)
        seqs = rng.randint(1, max(1, min(24, q_rows // 16 if train else q_rows)))
        k_rows = rng.choice([0, 0, _log_int(rng, 256 if train else 1, top)])
        return {k: v for k, v in _attend("", "train" if train else "forward", heads, kv_heads, dim,
                                         rng.random() < 0.7, seqs, q_rows, k_rows, cut).items() if k != "name"}
    if kind == "decode":
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 6, 8])
        seqs = _log_int(rng, 1, 48)
        room = _log_int(rng, 1, min(100000, 48 * 8192 * 8 * 128 // (seqs * kv_heads * 128)))
        return {k: v for k, v in _decode("", heads, kv_heads, rng.choice([64, 128]), seqs, rng.choice([1, 1, 1, 2, 5]),
                                         room, cut).items() if k != "name"}
    channels = 8 * _log_int(rng, 8, 1024)
    mode = "forward" if kind == "norm" else "train"
    stream, branch = (rng.choice(["bf16", "bf16", "f32"]) for _ in range(2))
    row_bytes = channels * 2 * sum({"bf16": 2, "f32": 4}[t] for t in (stream, branch)) * (2 if mode == "train" else 1)
    rows = _log_int(rng, 1, min(100000, 10**9 // row_bytes))
    # parameters in 32 bits are trained beside a residual stream in 32 bits
    param = "bf16" if (mode, stream) == ("train", "bf16") else rng.choice(["bf16", "f32"])
    return {k: v for k, v in _norm("", mode, rows, channels, rng.randint(1, min(12, rows)),
                                   rng.choice(["none", "rms", "layer"]), rng.choice(["rms", "layer"]), stream, branch,
                                   param, rng.random() < 0.6, cut).items() if k != "name"}


def _lengths(total, parts, cut):
    """`total` rows cut into `parts` sequences of very different lengths (empty ones among them)."""
    r = random.Random(cut)
    w = [math.exp(r.gauss(0.0, 1.2)) for _ in range(parts)]
    at = [0] + [round(total * sum(w[: i + 1]) / sum(w)) for i in range(parts)]
    return [b - a for a, b in zip(at, at[1:])]


def _lens_of(case):
    q = _lengths(case["q_rows"], case["seqs"], case["cut"])
    k = q if not case["k_rows"] else _lengths(case["k_rows"], case["seqs"], case["cut"] + 1)
    return q, k


def _used_of(case):
    r = random.Random(case["cut"])
    low = min(case["tokens"], case["room"])
    return [r.randint(max(low, case["room"] // 3), case["room"]) for _ in range(case["seqs"])]


def _offsets(lens, device):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=device)


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape, dtype=torch.bfloat16, gain=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device=dev) * gain + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "attend":
        ql, kl = _lens_of(case)
        nq, nk, d = sum(ql), sum(kl), case["dim"]
        s["q_offsets"] = _offsets(ql, dev)
        s["k_offsets"] = s["q_offsets"] if not case["k_rows"] else _offsets(kl, dev)
        s["q"] = randn(nq, case["heads"], d, gain=1.3)
        s["k"] = randn(nk, case["kv_heads"], d, gain=1.3)
        s["v"] = randn(nk, case["kv_heads"], d, mean=0.1)
        if case["pass"] == "train":
            s["dout"] = randn(nq, case["heads"], d)
    elif case["op"] == "decode":
        b, d = case["seqs"], case["dim"]
        s["q"] = randn(b, case["tokens"], case["heads"], d, gain=1.3)
        s["k"] = randn(b, case["room"], case["kv_heads"], d, gain=1.3)
        s["v"] = randn(b, case["room"], case["kv_heads"], d, mean=0.1)
        s["used"] = torch.tensor(_used_of(case), dtype=torch.int32, device=dev)
    else:
        n, c, b = case["rows"], case["channels"], case["seqs"]
        st, br, pa = (DTYPES[case[k]] for k in ("stream", "branch", "param"))
        s["offsets"] = _offsets(_lengths(n, b, case["cut"]), dev)
        loud = 1.0 + 6.0 * (torch.rand(c, generator=g, device=dev) < 0.02)    # a few loud channels, as residual streams have
        s["x"] = ((torch.randn(n, c, generator=g, device=dev) + 0.2) * loud).to(st)
        s["y"] = randn(n, c, dtype=br, gain=0.7)
        s["weight"] = randn(c, dtype=pa, gain=0.1, mean=1.0)
        s["post_weight"] = randn(c, dtype=pa, gain=0.1, mean=1.0) if case["post"] != "none" else None
        mods = case["mods"]
        s["gate"], s["scale"], s["shift"] = (randn(b, c, dtype=pa, gain=0.3) if mods else None for _ in range(3))
        if case["pass"] == "train":
            s["dh"] = randn(n, c, dtype=br)
            s["dx_out"] = randn(n, c, dtype=st)
    return s


ALPHA, EPS = 0.75, 1e-6


# ---- one pass ----------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "attend":
        return _plain_attend(s, case)
    if case["op"] == "decode":
        return _plain_decode(s, case)
    return _plain_norm(s, case)


def _run_own(s, case):
    from dynamic_block_sparse_variance_b200.packed import BlockNorm, PackedAttention

    if case["op"] == "attend":
        train = case["pass"] == "train"
        att = PackedAttention(case["heads"], case["kv_heads"], case["dim"], causal=case["causal"], training=train)
        o = att.forward(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"])
        if not train:
            return {"o": o, "lse": att.lse}
        dq, dk, dv = att.backward(s["dout"])
        return {"o": o, "lse": att.lse, "dq": dq, "dk": dk, "dv": dv}
    if case["op"] == "decode":
        att = PackedAttention(case["heads"], case["kv_heads"], case["dim"], causal=True, training=False)
        return {"o": att.forward(s["q"], s["k"], s["v"], k_used=s["used"]), "lse": att.lse}
    train = case["pass"] == "train"
    norm = BlockNorm(case["channels"], post=case["post"], pre=case["pre"], alpha=ALPHA, eps=EPS, training=train)
    x_out, h = norm.forward(s["x"], s["y"], offsets=s["offsets"], post_weight=s["post_weight"], gate=s["gate"],
                            weight=s["weight"], scale=s["scale"], shift=s["shift"])
    out = {"x_out": x_out, "h": h}
    if train:
        out.update((k, v) for k, v in norm.backward(s["dh"], s["dx_out"]).items() if v is not None)
    return out


# ---- plain forms -------------------------------------------------------------

def _softmax_rows(scores, seen):
    """Probabilities and log-sum-exp of masked rows; a row that sees nothing gets zeros and -inf."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    return p, (torch.log(total) + top).squeeze(-1)


def _plain_attend(s, case):
    hk, d, scale = case["kv_heads"], case["dim"], 1.0 / math.sqrt(case["dim"])
    g = case["heads"] // hk
    qo, ko = s["q_offsets"].long(), s["k_offsets"].long()
    nq, nk = s["q"].shape[0], s["k"].shape[0]
    iq, ik = torch.arange(nq, device=qo.device), torch.arange(nk, device=qo.device)
    sq, sk = torch.bucketize(iq, qo[1:], right=True), torch.bucketize(ik, ko[1:], right=True)
    seen = sq[:, None] == sk[None, :]
    if case["causal"]:      # the last row of a sequence's queries sees all of its keys
        seen &= (ik - ko[sk + 1])[None, :] <= (iq - qo[sq + 1])[:, None]
    q = s["q"].float().view(nq, hk, g, d).permute(1, 2, 0, 3)
    k, v = (s[n].float().permute(1, 0, 2)[:, None] for n in ("k", "v"))
    p, lse = _softmax_rows(torch.matmul(q, k.transpose(-1, -2)) * scale, seen)
    o = torch.matmul(p, v)
    back = lambda t: t.permute(2, 0, 1, 3).reshape(nq, hk * g, d).to(torch.bfloat16)
    out = {"o": back(o), "lse": lse.reshape(hk * g, nq)}
    if case["pass"] == "train":
        do = s["dout"].float().view(nq, hk, g, d).permute(1, 2, 0, 3)
        fold = lambda t: t.sum(1).permute(1, 0, 2).to(torch.bfloat16)
        out["dv"] = fold(torch.matmul(p.transpose(-1, -2), do))
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out["dq"] = back(torch.matmul(ds, k))
        out["dk"] = fold(torch.matmul(ds.transpose(-1, -2), q))
    return out


def _plain_decode(s, case):
    b, t, hq, d = s["q"].shape
    room, hk = s["k"].shape[1], s["k"].shape[2]
    q = s["q"].float().view(b, t, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    k, v = (s[n].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))
    at = torch.arange(room, device=q.device)
    last = s["used"].long()[:, None] - t + torch.arange(t, device=q.device)   # the last key each token sees
    seen = (at[None, None, :] <= last[:, :, None])[:, None, None]
    p, lse = _softmax_rows(torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d), seen)
    # rows of the cache that are not in use may hold anything
    v = v.masked_fill((at[None, :] >= s["used"].long()[:, None])[:, None, None, :, None], 0.0)
    o = torch.matmul(p, v).permute(0, 3, 1, 2, 4).reshape(b, t, hq, d).to(torch.bfloat16)
    return {"o": o, "lse": lse.permute(1, 2, 0, 3).reshape(hq, b * t)}


def _normed(x, kind):
    """x's rows normalised, and what they were divided by."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _normed_back(d, xhat, r, kind):
    if kind == "none":
        return d
    inner = d - xhat * (d * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        inner = inner - d.mean(-1, keepdim=True)
    return inner * r


def _plain_norm(s, case):
    x, y = s["x"].float(), s["y"].float()
    offs = s["offsets"].long()
    n, c = x.shape
    b = offs.numel() - 1
    of = torch.bucketize(torch.arange(n, device=x.device), offs[1:], right=True)
    w, w2 = s["weight"].float(), 1.0 if s["post_weight"] is None else s["post_weight"].float()
    gate, gain, shift = 1.0, 1.0, 0.0
    if case["mods"]:
        gate, gain, shift = s["gate"].float()[of], 1.0 + s["scale"].float()[of], s["shift"].float()[of]
    yhat, ry = _normed(y, case["post"])
    x_out = ALPHA * x + gate * (yhat * w2)
    xhat, rx = _normed(x_out, case["pre"])
    h = xhat * w * gain + shift
    out = {"x_out": x_out.to(s["x"].dtype), "h": h.to(s["y"].dtype)}
    if case["pass"] == "train":
        dh, dxo = s["dh"].float(), s["dx_out"].float()
        if x_out.dtype != out["x_out"].dtype:      # the backward starts from what the forward kept
            xhat, rx = _normed(out["x_out"].float(), case["pre"])
        pa = s["weight"].dtype      # a parameter's gradient has its type
        per = lambda t: torch.zeros(b, c, device=t.device).index_add_(0, of, t).to(pa)
        dr = _normed_back(dh * (w * gain), xhat, rx, case["pre"]) + dxo
        out["dx"] = (ALPHA * dr).to(s["x"].dtype)
        out["dy"] = _normed_back(dr * (gate * w2), yhat, ry, case["post"]).to(s["y"].dtype)
        out["dweight"] = (dh * xhat * gain).sum(0).to(pa)
        if s["post_weight"] is not None:
            out["dpost_weight"] = (dr * yhat * gate).sum(0).to(pa)
        if case["mods"]:
            out["dgate"], out["dscale"], out["dshift"] = per(dr * (yhat * w2)), per(dh * xhat * w), per(dh)
    return out


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    if case["op"] == "attend":
        ql, kl = _lens_of(case)
        pairs = 0
        for a, b in zip(ql, kl):
            if case["causal"]:
                # query i (from the end) sees b - i keys
                n = min(a, b)
                pairs += n * b - n * (n - 1) // 2
            else:
                pairs += a * b
        rows_q, rows_k = case["heads"] * sum(ql), case["kv_heads"] * sum(kl)
        train = case["pass"] == "train"
        # q, o (and dout, dq) and k, v (and dk, dv) once each, lse once
        return {"bytes": 2 * case["dim"] * (2 * rows_q + 2 * rows_k) * (2 if train else 1) + 4 * rows_q,
                "flops": (14 if train else 4) * case["dim"] * case["heads"] * pairs}
    if case["op"] == "decode":
        t, d = case["tokens"], case["dim"]
        used = _used_of(case)
        pairs = sum(max(0, u - i) for u in used for i in range(t))
        return {"bytes": 4 * d * case["kv_heads"] * sum(used) + case["heads"] * case["seqs"] * t * (4 * d + 4),
                "flops": 4 * d * case["heads"] * pairs}
    size = {"bf16": 2, "f32": 4}
    n, c, b, train = case["rows"], case["channels"], case["seqs"], case["pass"] == "train"
    # x, x_out, y, h; and dx_out, dx, dh, dy
    moved = n * c * 2 * (size[case["stream"]] + size[case["branch"]]) * (2 if train else 1)
    params = c * (1 + (case["post"] != "none") + (3 * b if case["mods"] else 0))
    return {"bytes": moved + params * size[case["param"]] * (2 if train else 1), "flops": n * c * (40 if train else 15)}


# ---- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "decode": _exact_decode, "norm": _exact_norm}[case["op"]](s, case)


def _one_sequence(q, k, v, seen, scale):
    """softmax(scale q k^T) v of one head in 64 bits, and its log-sum-exp."""
    z = (q @ k.T) * scale
    if seen is not None:
        z = torch.where(seen, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, dim=1)
    blind = torch.isinf(lse)
    p = torch.exp(z - torch.where(blind, torch.zeros_like(lse), lse)[:, None])
    return p, p @ v, lse


def _exact_attend(s, case):
    ql, kl = _lens_of(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    scale = d ** -0.5
    train = case["pass"] == "train"
    wide = lambda n: s[n].double()
    q, k, v = wide("q"), wide("k"), wide("v")
    out = {"o": torch.zeros_like(q), "lse": torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)}
    if train:
        do = wide("dout")
        out["dq"], out["dk"], out["dv"] = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = b = 0
    for nq, nk in zip(ql, kl):
        if nq and nk:
            seen = None
            if case["causal"]:
                seen = torch.ones(nq, nk, dtype=torch.bool, device=q.device).tril(nk - nq)
            for h in range(hq):
                j = h * hk // hq
                qh, kh, vh = q[a:a + nq, h], k[b:b + nk, j], v[b:b + nk, j]
                p, oh, lh = _one_sequence(qh, kh, vh, seen, scale)
                out["o"][a:a + nq, h] = oh
                out["lse"][h, a:a + nq] = lh
                if train:
                    doh = do[a:a + nq, h]
                    dp = doh @ vh.T
                    dz = p * (dp - (p * dp).sum(1, keepdim=True))
                    out["dv"][b:b + nk, j] += p.T @ doh
                    out["dq"][a:a + nq, h] = dz @ kh * scale
                    out["dk"][b:b + nk, j] += dz.T @ qh * scale
        a, b = a + nq, b + nk
    return out


def _exact_decode(s, case):
    q, k, v = s["q"].double(), s["k"], s["v"]
    b, t, hq, d = q.shape
    hk = k.shape[2]
    out = {"o": torch.zeros_like(q), "lse": torch.full((hq, b * t), -math.inf, dtype=torch.float64, device=q.device)}
    for i, n in enumerate(_used_of(case)):
        seen = torch.ones(t, n, dtype=torch.bool, device=q.device).tril(n - t)
        for h in range(hq):
            j = h * hk // hq
            _, o, lse = _one_sequence(q[i, :, h], k[i, :n, j].double(), v[i, :n, j].double(), seen, d ** -0.5)
            out["o"][i, :, h] = o
            out["lse"][h, i * t:(i + 1) * t] = lse
    return out


def _exact_norm(s, case):
    """The block by its definition, and its gradients by differentiation, both in 64 bits. A training pass
    differentiates the norm at the residual stream that the forward keeps (rounded to the stream's type)."""
    train = case["pass"] == "train"
    leaf = {n: s[n].double().requires_grad_(train) for n in ("x", "y", "weight", "post_weight", "gate", "scale", "shift")
            if s[n] is not None}
    lens = (s["offsets"][1:] - s["offsets"][:-1]).long()
    rows = lambda n: torch.repeat_interleave(leaf[n], lens, dim=0)

    def normalise(t, kind):
        if kind == "none":
            return t
        var = t.square().mean(1, keepdim=True) if kind == "rms" else t.var(1, keepdim=True, unbiased=False)
        return (t if kind == "rms" else t - t.mean(1, keepdim=True)) / torch.sqrt(var + EPS)

    branch = normalise(leaf["y"], case["post"])
    if "post_weight" in leaf:
        branch = branch * leaf["post_weight"]
    if case["mods"]:
        branch = branch * rows("gate")
    x_out = ALPHA * leaf["x"] + branch
    out = {"x_out": x_out.detach()}
    kept = x_out + (x_out.detach().to(s["x"].dtype).double() - x_out.detach()) if train else x_out

    def head(t):
        r = normalise(t, case["pre"]) * leaf["weight"]
        return r * (1.0 + rows("scale")) + rows("shift") if case["mods"] else r

    out["h"] = head(x_out).detach()
    if train:
        names = list(leaf)
        grads = torch.autograd.grad([head(kept), kept], [leaf[n] for n in names], [s["dh"].double(), s["dx_out"].double()])
        out.update(("d" + n, g) for n, g in zip(names, grads))
    return out
