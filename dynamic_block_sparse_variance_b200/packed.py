"""The dense layers and norms around the block-sparse one, over packed sequences.

PackedAttention  dense softmax attention over sequences of different lengths stored
                 one behind the other (self- or cross-attention, causal or not, grouped
                 heads), forward, backward, and single tokens over key/value caches.
BlockNorm        the norms before and after a block fused with its gate and the residual
                 stream, forward and backward; on its way it can give the norms ||y_n||
                 of the block's output that the sparse layer takes as its audio input.

PyTorch only allocates device memory and supplies the stream; each step is one call into
libprism_b200.so. Scratch is allocated per call on the current stream, so calls on several
streams and captured graphs share none of it. The checks of shapes and strides, and the
parameter block that follows from them, are kept per set of shapes and strides (a plan): a
small call is bound by the host, and its checks would cost more than its kernel.
"""

from __future__ import annotations

import torch

from . import prism as P

_KINDS = {"none": P.PRISM_NORM_NONE, "rms": P.PRISM_NORM_RMS, "layer": P.PRISM_NORM_LAYER}
_BF16 = torch.bfloat16
_raw_stream = torch._C._cuda_getCurrentRawStream      # of a device, without building a Stream object


def _need(ok, msg):
    if not ok:
        raise P.PrismError(P.PRISM_EINVAL, msg)


def _like(t):
    """A new contiguous tensor of t's shape and type (empty_like keeps the order of strides of a dense t)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


_plans = {}


def _plan(key, make):
    """The plan of `key` (nothing but shapes, strides, types and settings), made on first use."""
    p = _plans.get(key)
    if p is None:
        p = make()
        if len(_plans) >= 4096:
            _plans.clear()
        _plans[key] = p
    return p


def _same_device(index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise P.PrismError(P.PRISM_EINVAL, f"all tensors must be on device {index}, one is on {t.device}")


def _index(t, index, name):
    """A device array of int32: offsets or lengths. Its number of entries (-1: none)."""
    if t is None:
        return -1
    if not (t.dtype is torch.int32 and t.dim() == 1 and t.is_contiguous() and t.get_device() == index):
        raise P.PrismError(P.PRISM_EINVAL, f"{name} must be a contiguous int32 vector on device {index}")
    return t.shape[0]


def _heads_view(shape, stride, heads, dim, name):
    """(rows, sequences of a 4-D tensor or None, row stride, head stride) of [rows, heads, dim] or
    [sequences, rows, heads, dim]."""
    _need(len(shape) in (3, 4) and shape[-2] == heads and shape[-1] == dim,
          f"{name} must be [rows, {heads}, {dim}] or [sequences, rows, {heads}, {dim}], not {tuple(shape)}")
    _need(stride[-1] == 1, f"{name}: the elements of a head must be consecutive")
    head = stride[-2] if heads > 1 else dim
    if len(shape) == 3:
        n, seqs, row = shape[0], None, stride[0]
    else:
        seqs, per = shape[0], shape[1]
        n, row = seqs * per, stride[1] if per > 1 else stride[0]
        _need(seqs <= 1 or per <= 1 or stride[0] == per * stride[1], f"{name}: the sequences must lie one behind the other")
    if n <= 1:
        row = max(row, heads * head, dim)
        row += -row % 8
    _need(row > 0 and head > 0, f"{name}: expanded tensors are not taken")
    return n, seqs, row, head


def _used_here(at, stream, tensors):
    """The current raw stream of device `at`. Where it is not `stream`, the one that `tensors` were written on, the
    allocator learns that they are read here too: the next forward() lets go of them, maybe before this one is through."""
    now = _raw_stream(at)
    if now != stream:
        here = torch.cuda.current_stream(at)
        for t in tensors:
            if t is not None:
                t.record_stream(here)
    return now


class _FwdPlan:
    __slots__ = ("p", "q_rows", "ws", "offsets")


class PackedAttention:
    """Dense attention over packed sequences.

    Tensors are [rows, heads, head_dim] bf16 with the sequences' rows one behind the other and
    ``q_offsets`` / ``k_offsets`` (device int32, sequences + 1 entries), or [sequences, rows, heads,
    head_dim] without offsets; strided slices of larger tensors are taken as they are. Query head h reads
    key/value head h // (heads // kv_heads). With ``causal`` the last query of a sequence sees all of its
    keys, the one before it all but the last, and so on; a query that sees no key gets 0 (and lse -inf).
    ``k_used`` (device int32): only so many of each sequence's key rows are in use, as in a cache with room.
    With ``training`` forward() keeps what backward() needs: its inputs and outputs (not copies; leave
    them unchanged until then) and the rounding residual of O. No output may overlap an input. Rows outside every sequence are left as
    they were; pass ``out`` (and dq, dk, dv) to say what that is. Calls run on the device of q and its
    current stream.
    """

    def __init__(self, heads, kv_heads=None, head_dim=128, *, causal=True, scale=0.0, training=True):
        self.heads, self.kv_heads, self.head_dim = heads, heads if kv_heads is None else kv_heads, head_dim
        self.causal, self.scale, self.training = causal, scale, training
        self.lse = None
        self._saved = None

    def _forward_plan(self, q, k, v, o, n_qo, n_ko, n_used):
        """Plan of a forward call from (shape, stride) pairs (o None: contiguous) and the numbers of offsets."""
        d = self.head_dim
        q_rows, q_seqs, *q_st = _heads_view(*q, self.heads, d, "q")
        k_rows, k_seqs, *k_st = _heads_view(*k, self.kv_heads, d, "k")
        v_st = _heads_view(*v, self.kv_heads, d, "v")[2:]
        _need(k[0] == v[0], "k and v must have the same shape")
        _need(q_seqs is None or n_qo < 0, "q_offsets belong to a 3-D q")
        _need(k_seqs is None or n_ko < 0, "k_offsets belong to 3-D k and v")
        counts = {n for n in (q_seqs, k_seqs, n_qo - 1 if n_qo >= 0 else None, n_ko - 1 if n_ko >= 0 else None,
                              n_used if n_used >= 0 else None) if n is not None}
        _need(len(counts) <= 1, f"q, k, offsets and k_used speak of different numbers of sequences: {sorted(counts)}")
        seqs = counts.pop() if counts else 1
        _need(seqs >= 0, "offsets have one entry more than there are sequences")
        plan = _FwdPlan()
        plan.offsets = seqs > 0
        if seqs == 0:       # no sequences: no rows
            seqs = 1
            _need(q_rows == 0 and k_rows == 0, "rows without sequences")
        p = plan.p = P.prism_packed_params(seqs=seqs, heads=self.heads, kv_heads=self.kv_heads, head_dim=d, q_rows=q_rows,
                                           k_rows=k_rows, causal=int(self.causal), scale=self.scale)
        p.q_stride[:], p.k_stride[:], p.v_stride[:] = q_st, k_st, v_st
        if o is not None:
            p.o_stride[:] = _heads_view(q[0], o, self.heads, d, "out")[2:]
        plan.q_rows = q_rows
        plan.ws = P.prism_packed_workspace_size(p, P.PRISM_WS_PACKED_FWD)
        return plan

    def forward(self, q, k, v, q_offsets=None, k_offsets=None, *, k_used=None, out=None):
        """O, shaped like q. ``self.lse`` [heads, rows of q] is its log-sum-exp. Without ``k_offsets`` a 3-D k
        has the offsets of q."""
        at = q.get_device()
        _need(at >= 0, "packed attention runs on a CUDA device")
        if at != torch.cuda.current_device():
            with torch.cuda.device(at):
                return self.forward(q, k, v, q_offsets, k_offsets, k_used=k_used, out=out)
        if not (q.dtype is _BF16 and k.dtype is _BF16 and v.dtype is _BF16 and (out is None or out.dtype is _BF16)):
            raise TypeError("q, k, v and out must be bfloat16")
        _same_device(at, k, v, out)
        if k_offsets is None and k.dim() == 3:
            k_offsets = q_offsets
        n_qo, n_used = _index(q_offsets, at, "q_offsets"), _index(k_used, at, "k_used")
        n_ko = n_qo if k_offsets is q_offsets else _index(k_offsets, at, "k_offsets")
        qs, ks, vs = (q.shape, q.stride()), (k.shape, k.stride()), (v.shape, v.stride())
        if out is not None:
            _need(out.shape == q.shape, "out must have the shape of q")
            os = out.stride()
        else:
            os = None
        key = (self.heads, self.kv_heads, self.head_dim, self.causal, self.scale, qs, ks, vs, os, n_qo, n_ko, n_used)
        plan = _plan(key, lambda: self._forward_plan(qs, ks, vs, os, n_qo, n_ko, n_used))
        if not plan.offsets:
            q_offsets = k_offsets = k_used = None
        if out is None:
            out = _like(q)
        lse = q.new_empty((self.heads, plan.q_rows), dtype=torch.float32)
        o_res = q.new_empty((plan.q_rows, self.heads, self.head_dim)) if self.training else None
        ws = q.new_empty(plan.ws, dtype=torch.uint8) if plan.ws else None
        stream = _raw_stream(at)
        P.prism_packed_attn_fwd(plan.p, q, k, v, q_offsets, k_offsets, k_used, out, o_res, lse, ws, stream)
        self.lse = lse
        self._saved = (key, plan.p, stream, q, k, v, out, o_res, lse, q_offsets, k_offsets, k_used) if self.training else None
        return out

    def _backward_plan(self, p, shapes, strides):
        p = type(p).from_buffer_copy(p)
        for name, shape, st, heads in zip(("dout", "dq", "dk", "dv"), shapes, strides,
                                          (self.heads, self.heads, self.kv_heads, self.kv_heads)):
            if st is not None:
                getattr(p, name + "_stride")[:] = _heads_view(shape, st, heads, self.head_dim, name)[2:]
        return p, P.prism_packed_workspace_size(p, P.PRISM_WS_PACKED_BWD)

    def backward(self, dout, dq=None, dk=None, dv=None):
        """Gradients (dQ, dK, dV) of the last forward(), shaped like q, k and v."""
        _need(self._saved is not None, "backward() needs a forward() with training=True before it")
        key, p, stream, q, k, v, o, o_res, lse, q_offsets, k_offsets, k_used = self._saved
        at = q.get_device()
        if at != torch.cuda.current_device():
            with torch.cuda.device(at):
                return self.backward(dout, dq, dk, dv)
        _need(dout.shape == q.shape, "dout must have the shape of q")
        _same_device(at, dout, dq, dk, dv)
        strides = [dout.stride()]
        for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            _need(g is None or g.shape == like.shape, f"{name} must have the shape of its input")
            strides.append(None if g is None else g.stride())
        for g in (dout, dq, dk, dv):
            if g is not None and g.dtype is not _BF16:
                raise TypeError("dout, dq, dk and dv must be bfloat16")
        bp, n = _plan((key, *strides), lambda: self._backward_plan(p, (q.shape, q.shape, k.shape, v.shape), strides))
        dq = _like(q) if dq is None else dq
        dk = _like(k) if dk is None else dk
        dv = _like(v) if dv is None else dv
        ws = q.new_empty(n, dtype=torch.uint8) if n else None
        here = _used_here(at, stream, self._saved[3:])
        P.prism_packed_attn_bwd(bp, q, k, v, o, o_res, dout, lse, q_offsets, k_offsets, k_used, dq, dk, dv, ws, here)
        return dq, dk, dv


def _norm_rows(shape, stride, channels, name):
    """Row stride of a [rows, channels] or [sequences, rows, channels] tensor (0: contiguous)."""
    rows = stride[-2] if len(shape) == 2 or shape[1] > 1 else stride[0]
    n = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    _need(stride[-1] == 1, f"{name}: the elements of a row must be consecutive")
    if n <= 1:
        return 0
    _need(len(shape) == 2 or shape[0] <= 1 or shape[1] <= 1 or stride[0] == shape[1] * stride[1],
          f"{name}: the sequences must lie one behind the other")
    _need(rows >= channels, f"{name}: expanded tensors are not taken")
    return rows


def _on(out, kept):
    """Whether an output takes the place of a tensor."""
    return out is not None and kept is not None and out.data_ptr() == kept.data_ptr() and out.numel() > 0


def _keep(x, y, x_out, h):
    """Refuses the in-place forms that overwrite what the backward of a training forward starts from: y, and x
    where there is no y."""
    if y is None:
        _need(not _on(h, x), "h must not take the place of x, which backward() needs where there is no y")
    else:
        _need(not _on(h, y), "h must not take the place of y, which backward() needs")
        _need(not _on(x_out, y), "x_out must not take the place of y, which backward() needs")


class _NormPlan:
    __slots__ = ("p", "ws", "branch")


_FLOATS = {torch.bfloat16: P.PRISM_BF16, torch.float32: P.PRISM_F32}
_PARAMS = ("post_weight", "gate", "weight", "scale", "shift")


def _layout(t):
    return None if t is None else (t.shape, t.stride(), t.dtype)


class BlockNorm:
    """The norms around a block:

        x_out = alpha x + gate (N_post(y) post_weight)
        h     = N_pre(x_out) weight (1 + scale) + shift

    ``post`` is "none", "rms" or "layer", ``pre`` "rms" or "layer". x (the residual stream) and y (the
    block's output) are [rows, channels] or [sequences, rows, channels], bf16 or f32 each; the weights are
    [channels], gate, scale and shift [channels] or [1, channels] (shared), or [sequences, channels] with
    ``offsets`` saying which rows are whose; all of these have one type, bf16 or f32. Every parameter may be
    left out. With ``training`` forward() keeps what backward() needs: y, x_out and the parameters (not copies; leave
    them unchanged until then). Outputs may take the place of inputs of the same type and strides: x_out that of x, dx
    that of dx_out, dy that of dh and, without training, h that of y or x and x_out that of y. A backward() whose dx or
    dy takes the place of what it starts from is the last one of its forward(). Rows outside every sequence are left as they were. Calls run on the device of x and its current stream.
    """

    def __init__(self, channels, *, post="none", pre="rms", eps=1e-6, alpha=1.0, training=True):
        _need(post in _KINDS and pre in _KINDS, f"norms are one of {sorted(_KINDS)}")
        self.channels, self.post, self.pre = channels, post, pre
        self.eps, self.alpha, self.training = eps, alpha, training
        self._saved = None

    def _forward_plan(self, x, y, x_out, h, h_dtype, n_off, params):
        c = self.channels
        for t in (x, y):
            if t is not None and t[2] not in _FLOATS:
                raise TypeError(f"unsupported dtype {t[2]}")
        shape = x[0]
        _need(len(shape) in (2, 3) and shape[-1] == c,
              f"x must be [rows, {c}] or [sequences, rows, {c}], not {tuple(shape)}")
        branch = y[2] if y is not None else h[2] if h is not None else h_dtype or x[2]
        if branch not in _FLOATS:
            raise TypeError(f"unsupported dtype {branch}")
        for name, t, dtype in (("y", y, None), ("x_out", x_out, x[2]), ("h", h, branch)):
            if t is not None:
                _need(t[0] == shape, f"{name} must have the shape {tuple(shape)}, not {tuple(t[0])}")
                if dtype is not None and t[2] != dtype:
                    raise TypeError(f"{name} must be {dtype}, not {t[2]}")
        given = {n: t for n, t in zip(_PARAMS, params) if t is not None}
        per = [t[0][0] for n, t in given.items() if len(t[0]) == 2 and t[0][0] > 1]
        rows = shape[0] if len(shape) == 2 else shape[0] * shape[1]
        if n_off >= 0:
            _need(len(shape) == 2, "offsets belong to a 2-D x")
            seqs = n_off - 1
            _need(seqs >= 1, "offsets have one entry more than there are sequences, of which there is one at least")
        else:
            seqs = max(1, shape[0] if len(shape) == 3 else per[0] if per else 1)
        types = {t[2] for t in given.values()}
        _need(len(types) <= 1, "weights, gate, scale and shift must have one type")
        if types and not types <= set(_FLOATS):
            raise TypeError(f"unsupported dtype {types.pop()}")
        plan = _NormPlan()
        plan.branch = branch
        p = plan.p = P.prism_norm_params(rows=rows, channels=c, seqs=seqs, stream_dtype=_FLOATS[x[2]],
                                         branch_dtype=_FLOATS[branch], param_dtype=_FLOATS[types.pop()] if types else P.PRISM_F32,
                                         post_norm=_KINDS[self.post], pre_norm=_KINDS[self.pre], eps=self.eps, alpha=self.alpha)
        for name, (ps, st, _) in given.items():
            _need(ps[-1] == c and (len(ps) == 1 or (len(ps) == 2 and "weight" not in name and ps[0] in (1, seqs))),
                  f"{name} has the shape {tuple(ps)}")
            _need(st[-1] == 1, f"{name}: the elements of a row must be consecutive")
            if len(ps) == 2 and ps[0] > 1:
                _need(st[0] >= c, f"{name}: expanded tensors are not taken; pass [channels]")
                setattr(p, name + "_stride", st[0])
        for name, t in (("x", x), ("y", y), ("x_out", x_out), ("h", h)):
            if t is not None:
                setattr(p, name + "_row_stride", _norm_rows(t[0], t[1], c, name))
        if y is None:
            p.x_out_row_stride = p.x_row_stride      # the backward's x_out is x
        plan.ws = P.prism_block_norm_workspace_size(p)
        return plan

    def forward(self, x, y=None, *, offsets=None, post_weight=None, gate=None, weight=None, scale=None, shift=None,
                x_out=None, h=None, y_norms=None, h_dtype=None):
        """(x_out, h). Without y: (x, N_pre(x) weight (1 + scale) + shift). ``y_norms`` (float [rows]) receives
        the Euclidean norms of y's rows; ``h_dtype`` is the type of h where there is no y (default: x's)."""
        at = x.get_device()
        _need(at >= 0, "block norms run on a CUDA device")
        if at != torch.cuda.current_device():
            with torch.cuda.device(at):
                return self.forward(x, y, offsets=offsets, post_weight=post_weight, gate=gate, weight=weight, scale=scale,
                                    shift=shift, x_out=x_out, h=h, y_norms=y_norms, h_dtype=h_dtype)
        params = (post_weight, gate, weight, scale, shift)
        _same_device(at, y, x_out, h, y_norms, *params)
        n_off = _index(offsets, at, "offsets")
        _need(y is not None or x_out is None, "x_out belongs to a y")
        if self.training:
            _keep(x, y, x_out, h)
        layouts = (_layout(x), _layout(y), _layout(x_out), _layout(h), h_dtype, n_off,
                   (_layout(post_weight), _layout(gate), _layout(weight), _layout(scale), _layout(shift)))
        key = (self.channels, self.post, self.pre, self.eps, self.alpha, layouts)
        plan = _plan(key, lambda: self._forward_plan(*layouts))
        if y is not None and x_out is None:
            x_out = _like(x)
        if h is None:
            h = _like(x) if plan.branch is x.dtype else x.new_empty(x.shape, dtype=plan.branch)
        if y_norms is not None:
            _need(y_norms.dtype == torch.float32 and y_norms.is_contiguous() and y_norms.numel() == plan.p.rows,
                  f"y_norms must be {plan.p.rows} contiguous floats")
        stream = _raw_stream(at)
        P.prism_block_norm_fwd(plan.p, x, y, offsets, post_weight, gate, weight, scale, shift, x_out, h, y_norms, stream)
        kept = x if y is None else x_out
        self._saved = (key, plan, stream, kept, y, offsets, params) if self.training else None
        return kept, h

    def _backward_plan(self, plan, kept, y, given):
        p = type(plan.p).from_buffer_copy(plan.p)
        stream = next(t for t, n in _FLOATS.items() if n == p.stream_dtype)
        for name, t, dtype in zip(("dh", "dx_out", "dx", "dy"), given, (plan.branch, stream, stream, plan.branch)):
            if t is None:
                continue
            if t[2] != dtype:
                raise TypeError(f"{name} must be {dtype}, not {t[2]}")
            _need(t[0] == kept, f"{name} must have the shape {tuple(kept)}, not {tuple(t[0])}")
            setattr(p, name + "_row_stride", _norm_rows(t[0], t[1], self.channels, name))
        return p

    def backward(self, dh, dx_out=None, dx=None, dy=None):
        """Gradients of the last forward(): a dict of dx, dy and the parameters' (None for what was left out),
        shaped and typed like what they belong to. ``dx_out``: the gradient that reaches the residual stream behind
        the block (None: zero)."""
        _need(self._saved is not None, "backward() needs a forward() with training=True before it")
        key, plan, stream, kept, y, offsets, params = self._saved
        at = kept.get_device()
        if at != torch.cuda.current_device():
            with torch.cuda.device(at):
                return self.backward(dh, dx_out, dx, dy)
        _same_device(at, dh, dx_out, dx, dy)
        given = (_layout(dh), _layout(dx_out), _layout(dx), None if y is None else _layout(dy))
        p = _plan((key, given), lambda: self._backward_plan(plan, kept.shape, y, given))
        if dx is None:
            dx = _like(kept)
        if y is None:
            dy = None
        elif dy is None:
            dy = _like(y)
        post_weight, gate, weight, scale, shift = params
        grads = [None if t is None or (y is None and i < 2) else _like(t) for i, t in enumerate(params)]
        ws = kept.new_empty(plan.ws, dtype=torch.uint8)
        here = _used_here(at, stream, (kept, y, offsets, *params))
        P.prism_block_norm_bwd(p, kept, y, offsets, post_weight, gate, weight, scale, dh, dx_out, dx, dy, *grads, ws, here)
        if _on(dx, kept) or _on(dx, y) or _on(dy, kept) or _on(dy, y):
            self._saved = None
        return {"dx": dx, "dy": dy, **{"d" + n: g for n, g in zip(_PARAMS, grads)}}
