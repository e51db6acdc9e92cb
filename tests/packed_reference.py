"""Plain 64-bit references of the packed-sequence operators (numpy, sequence by sequence and head by head),
with the error bounds that the kernels' roundings allow."""

import numpy as np

U = 2.0 ** -8          # a bf16 rounding is off by at most this, relative to the value (half a step)
TINY = 2.0 ** -100


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def attention(q, k, v, q_off, k_off, causal, scale, used=None, dout=None):
    """o, lse and, with dout, dq, dk, dv; and bounds of their errors, elementwise (with dout: a third dict).

    Bounds, with p the probabilities, a = p |v| and D the row sum of dout o:
      o    the probabilities enter the product with v rounded once (U a), the result is rounded once (U |o|)
      dv   likewise: U p^T |dout| + U |dv|
      ds   D comes from the computed o, whose products' error is U a: |dD| <= U |dout| . a; ds is rounded once
           as an operand: U |ds| + p |dD|; dq and dk sum that times |k| or |q| and are rounded once
    Sums in 32 bits, exponentials and the 16-bit residual of o add relative errors near 2^-16: covered by a
    factor of 1.1 and by `slack` = 2^-14 of the same sums of magnitudes.
    The part of the bounds that is such sums alone comes third: dP and D sum 128 products each, so dS is off by up to
    2 x 128 x 2^-24 = 2^-16 of p (|dout| |v| + |dout| a) however small it is (exactly 0 where a row sees one key).
    """
    hq, hk = q.shape[1], k.shape[1]
    o, lse = np.zeros_like(q), np.full((hq, q.shape[0]), -np.inf)
    bo = np.zeros_like(q)
    g = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    bg, rest = ({n: np.zeros_like(x) for n, x in g.items()} for _ in range(2))
    slack = 2.0 ** -14
    for b in range(len(q_off) - 1):
        q0, lq = q_off[b], q_off[b + 1] - q_off[b]
        k0, lk = k_off[b], k_off[b + 1] - k_off[b]
        if used is not None:
            lk = used[b]
        if lq == 0 or lk == 0:
            continue
        seen = np.ones((lq, lk), bool)
        if causal:
            seen = np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq
        for h in range(hq):
            j = h // (hq // hk)
            Q, K, V = q[q0:q0 + lq, h], k[k0:k0 + lk, j], v[k0:k0 + lk, j]
            z = np.where(seen, scale * (Q @ K.T), -np.inf)
            m = z.max(1, keepdims=True)
            e = np.where(seen, np.exp(z - np.where(np.isfinite(m), m, 0.0)), 0.0)
            l = e.sum(1, keepdims=True)
            p = e / np.where(l > 0, l, 1.0)
            O, a = p @ V, p @ np.abs(V)
            o[q0:q0 + lq, h] = O
            bo[q0:q0 + lq, h] = 1.1 * U * (a + np.abs(O)) + slack * a
            with np.errstate(divide="ignore"):
                lse[h, q0:q0 + lq] = (np.log(l) + np.where(np.isfinite(m), m, 0.0))[:, 0]
            if dout is None:
                continue
            G = dout[q0:q0 + lq, h]
            dp = G @ V.T
            D = (G * O).sum(1, keepdims=True)
            ds = p * (dp - D)
            mag = np.abs(G) @ np.abs(V).T + (np.abs(G) * a).sum(1, keepdims=True)
            eds = 1.1 * U * (np.abs(ds) + p * (np.abs(G) * a).sum(1, keepdims=True)) + slack * p * mag
            g["dq"][q0:q0 + lq, h] = scale * ds @ K
            g["dk"][k0:k0 + lk, j] += scale * ds.T @ Q
            g["dv"][k0:k0 + lk, j] += p.T @ G
            rest["dq"][q0:q0 + lq, h] = scale * 2.0 ** -16 * (p * mag) @ np.abs(K)
            rest["dk"][k0:k0 + lk, j] += scale * 2.0 ** -16 * (p * mag).T @ np.abs(Q)
            bg["dq"][q0:q0 + lq, h] = scale * eds @ np.abs(K)
            bg["dk"][k0:k0 + lk, j] += scale * eds.T @ np.abs(Q)
            bg["dv"][k0:k0 + lk, j] += (1.1 * U + slack) * p.T @ np.abs(G)
    for n in g:
        bg[n] += 1.1 * U * np.abs(g[n])
    out = dict(o=o, lse=lse)
    bounds = dict(o=bo + TINY, lse=2e-5 * np.where(np.isfinite(lse), 1.0 + np.abs(lse), 1.0))
    if dout is not None:
        out.update(g)
        bounds.update({n: x + TINY for n, x in bg.items()})
    return (out, bounds) if dout is None else (out, bounds, rest)


def _normed(z, kind, eps):
    if kind == "none":
        return z, np.ones((len(z), 1))
    c = z - z.mean(1, keepdims=True) if kind == "layer" else z
    r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    return c * r, r


def _normed_back(d, zhat, r, kind):
    if kind == "none":
        return d
    out = d - zhat * (d * zhat).mean(1, keepdims=True)
    if kind == "layer":
        out = out - d.mean(1, keepdims=True)
    return out * r


def block_norm(x, y, off, post, pre, eps, alpha, post_weight=None, gate=None, weight=None, scale=None, shift=None,
               dh=None, dx_out=None, kept=None):
    """x_out, h, y_norms and, with dh, the gradients; all arrays float64. gate, scale, shift: [sequences, C] or
    [1, C]; rows outside the sequences are returned as zeros. ``kept``: x_out as the forward kept it."""
    n, c = x.shape
    seq = np.full(n, -1)
    for b in range(len(off) - 1):
        seq[off[b]:off[b + 1]] = b
    inside = seq >= 0
    of = np.where(inside, seq, 0)

    def rows(t, default):
        return np.full((1, c), default) if t is None else (t[of] if len(t) > 1 else t)

    w, w2 = (np.ones(c) if t is None else t for t in (weight, post_weight))
    G, S, B = rows(gate, 1.0), 1.0 + rows(scale, 0.0), rows(shift, 0.0)
    out = {}
    if y is not None:
        yh, ry = _normed(y, post, eps)
        x_out = alpha * x + G * (yh * w2)
        out["x_out"] = x_out * inside[:, None]
        out["y_norms"] = np.sqrt((y * y).sum(1)) * inside
    else:
        x_out, alpha = x, 1.0
    out["h"] = (_normed(x_out, pre, eps)[0] * w * S + B) * inside[:, None]
    if dh is None:
        return out
    xh, rx = _normed(x_out if kept is None else kept, pre, eps)
    dr = _normed_back(dh * w * S, xh, rx, pre) + (0.0 if dx_out is None else dx_out)
    out["dx"] = alpha * dr * inside[:, None]

    def per(t, shared):
        r = np.zeros((len(off) - 1, c))
        np.add.at(r, seq[inside], t[inside])
        return r.sum(0, keepdims=True) if shared else r

    def is_shared(t):
        return t is not None and len(t) == 1

    out["dweight"] = (dh * xh * S)[inside].sum(0)
    out["dscale"] = per(dh * xh * w, is_shared(scale))
    out["dshift"] = per(dh, is_shared(shift))
    if y is not None:
        out["dy"] = _normed_back(dr * (G * w2), yh, ry, post) * inside[:, None]
        out["dpost_weight"] = (dr * yh * G)[inside].sum(0)
        out["dgate"] = per(dr * yh * w2, is_shared(gate))
        # magnitudes of the sums, for bounds
        out["abs"] = dict(dpost_weight=np.abs(dr * yh * G)[inside].sum(0), dgate=per(np.abs(dr * yh * w2), is_shared(gate)))
    else:
        out["abs"] = {}
    out["abs"].update(dweight=np.abs(dh * xh * S)[inside].sum(0), dscale=per(np.abs(dh * xh * w), is_shared(scale)),
                      dshift=per(np.abs(dh), is_shared(shift)))
    return out
