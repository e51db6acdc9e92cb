"""The dense layers and norms around the block-sparse one, over packed sequences.

PackedAttention  dense softmax attention over sequences of different lengths stored
                 one behind the other (self- or cross-attention, causal or not, grouped
                 heads), forward, backward, and single tokens over key/value caches.
BlockNorm        the norms before and after a block fused with its gate and the residual
                 stream, forward and backward; on its way it can give the norms ||y_n||
                 of the block's output that the sparse layer takes as its audio input.

PyTorch only allocates device memory and supplies the stream; each step is one call into
libprism_b200.so. Scratch is allocated per call on the current stream, so calls on several
streams and captured graphs share none of it.
"""

from __future__ import annotations

import torch

from . import prism as P

_KINDS = {"none": P.PRISM_NORM_NONE, "rms": P.PRISM_NORM_RMS, "layer": P.PRISM_NORM_LAYER}


def _need(ok, msg):
    if not ok:
        raise P.PrismError(P.PRISM_EINVAL, msg)


class _on_device:
    """Makes `dev` the current device for the calls inside (nothing to do if it is already)."""

    def __init__(self, dev):
        self.guard = torch.cuda.device(dev) if dev.index != torch.cuda.current_device() else None

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


def _index(t, n, dev, name):
    """A device array of int32: offsets or lengths."""
    if t is not None:
        _need(t.dtype == torch.int32 and t.dim() == 1 and t.is_contiguous() and t.device == dev,
              f"{name} must be a contiguous int32 vector on {dev}")
        _need(n is None or t.numel() == n, f"{name} must have {n} entries, not {t.numel()}")
    return t


def _heads_view(t, heads, dim, dev, name):
    """(rows, sequences of a 4-D tensor or None, row stride, head stride) of [rows, heads, dim] or
    [sequences, rows, heads, dim] bf16."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    _need(t.device == dev, f"{name} is on {t.device}, not {dev}")
    _need(t.dim() in (3, 4) and t.shape[-2] == heads and t.shape[-1] == dim,
          f"{name} must be [rows, {heads}, {dim}] or [sequences, rows, {heads}, {dim}], not {tuple(t.shape)}")
    st = t.stride()
    _need(st[-1] == 1, f"{name}: the elements of a head must be consecutive")
    head = st[-2] if heads > 1 else dim
    if t.dim() == 3:
        n, seqs, row = t.shape[0], None, st[0]
    else:
        seqs, per = t.shape[0], t.shape[1]
        n, row = seqs * per, st[1] if per > 1 else st[0]
        _need(seqs <= 1 or per <= 1 or st[0] == per * st[1], f"{name}: the sequences must lie one behind the other")
    if n <= 1:
        row = max(row, heads * head, dim)
        row += -row % 8
    _need(row > 0 and head > 0, f"{name}: expanded tensors are not taken")
    return n, seqs, row, head


class PackedAttention:
    """Dense attention over packed sequences.

    Tensors are [rows, heads, head_dim] bf16 with the sequences' rows one behind the other and
    ``q_offsets`` / ``k_offsets`` (device int32, sequences + 1 entries), or [sequences, rows, heads,
    head_dim] without offsets; strided slices of larger tensors are taken as they are. Query head h reads
    key/value head h // (heads // kv_heads). With ``causal`` the last query of a sequence sees all of its
    keys, the one before it all but the last, and so on; a query that sees no key gets 0 (and lse -inf).
    ``k_used`` (device int32): only so many of each sequence's key rows are in use, as in a cache with room.
    With ``training`` forward() keeps what backward() needs: its inputs and outputs (not copies; leave
    them unchanged until then) and the rounding residual of O. Rows outside every sequence are left as
    they were; pass ``out`` (and dq, dk, dv) to say what that is.
    """

    def __init__(self, heads, kv_heads=None, head_dim=128, *, causal=True, scale=0.0, training=True):
        self.heads, self.kv_heads, self.head_dim = heads, heads if kv_heads is None else kv_heads, head_dim
        self.causal, self.scale, self.training = causal, scale, training
        self.lse = None
        self._saved = None

    def _params(self, seqs, q_rows, k_rows):
        return P.prism_packed_params(seqs=seqs, heads=self.heads, kv_heads=self.kv_heads, head_dim=self.head_dim,
                                     q_rows=q_rows, k_rows=k_rows, causal=int(self.causal), scale=self.scale)

    def _workspace(self, p, kind, dev):
        n = P.prism_packed_workspace_size(p, kind)
        return torch.empty(n, dtype=torch.uint8, device=dev) if n else None

    def forward(self, q, k, v, q_offsets=None, k_offsets=None, *, k_used=None, out=None):
        """O, shaped like q. ``self.lse`` [heads, rows of q] is its log-sum-exp. Without ``k_offsets`` a 3-D k
        has the offsets of q."""
        dev, d = q.device, self.head_dim
        _need(dev.type == "cuda", "packed attention runs on a CUDA device")
        q_rows, q_seqs, *q_st = _heads_view(q, self.heads, d, dev, "q")
        k_rows, k_seqs, *k_st = _heads_view(k, self.kv_heads, d, dev, "k")
        v_rows, v_seqs, *v_st = _heads_view(v, self.kv_heads, d, dev, "v")
        _need(k.shape == v.shape, "k and v must have the same shape")
        if k_offsets is None and k_seqs is None:
            k_offsets = q_offsets
        _need(q_seqs is None or q_offsets is None, "q_offsets belong to a 3-D q")
        _need(k_seqs is None or k_offsets is None, "k_offsets belong to 3-D k and v")
        counts = {n for n in (q_seqs, k_seqs, None if q_offsets is None else q_offsets.numel() - 1,
                              None if k_offsets is None else k_offsets.numel() - 1,
                              None if k_used is None else k_used.numel()) if n is not None}
        _need(len(counts) <= 1, f"q, k, offsets and k_used speak of different numbers of sequences: {sorted(counts)}")
        seqs = counts.pop() if counts else 1
        if seqs == 0:
            seqs = 1        # no sequences: no rows
            _need(q_rows == 0 and k_rows == 0, "rows without sequences")
            q_offsets = k_offsets = k_used = None
        _index(q_offsets, seqs + 1, dev, "q_offsets")
        _index(k_offsets, seqs + 1, dev, "k_offsets")
        _index(k_used, seqs, dev, "k_used")
        p = self._params(seqs, q_rows, k_rows)
        p.q_stride[:], p.k_stride[:], p.v_stride[:] = q_st, k_st, v_st
        with _on_device(dev):
            if out is None:
                out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
            else:
                _need(out.shape == q.shape, "out must have the shape of q")
            p.o_stride[:] = _heads_view(out, self.heads, d, dev, "out")[2:]
            lse = torch.empty(self.heads, q_rows, dtype=torch.float32, device=dev)
            o_res = torch.empty(q_rows, self.heads, d, dtype=torch.bfloat16, device=dev) if self.training else None
            P.prism_packed_attn_fwd(p, q, k, v, q_offsets, k_offsets, k_used, out, o_res, lse,
                                    self._workspace(p, P.PRISM_WS_PACKED_FWD, dev))
        self.lse = lse
        self._saved = (p, q, k, v, out, o_res, lse, q_offsets, k_offsets, k_used) if self.training else None
        return out

    def backward(self, dout, dq=None, dk=None, dv=None):
        """Gradients (dQ, dK, dV) of the last forward(), shaped like q, k and v."""
        _need(self._saved is not None, "backward() needs a forward() with training=True before it")
        p, q, k, v, o, o_res, lse, q_offsets, k_offsets, k_used = self._saved
        dev, d = q.device, self.head_dim
        _need(dout.shape == q.shape, "dout must have the shape of q")
        with _on_device(dev):
            grads = []
            for given, like, heads, name in ((dq, q, self.heads, "dq"), (dk, k, self.kv_heads, "dk"),
                                             (dv, v, self.kv_heads, "dv")):
                g = torch.empty(like.shape, dtype=torch.bfloat16, device=dev) if given is None else given
                _need(g.shape == like.shape, f"{name} must have the shape of its input")
                getattr(p, name + "_stride")[:] = _heads_view(g, heads, d, dev, name)[2:]
                grads.append(g)
            p.dout_stride[:] = _heads_view(dout, self.heads, d, dev, "dout")[2:]
            P.prism_packed_attn_bwd(p, q, k, v, o, o_res, dout, lse, q_offsets, k_offsets, k_used, *grads,
                                    self._workspace(p, P.PRISM_WS_PACKED_BWD, dev))
        return tuple(grads)


class BlockNorm:
    """The norms around a block:

        x_out = alpha x + gate (N_post(y) post_weight)
        h     = N_pre(x_out) weight (1 + scale) + shift

    ``post`` is "none", "rms" or "layer", ``pre`` "rms" or "layer". x (the residual stream) and y (the
    block's output) are [rows, channels] or [sequences, rows, channels], bf16 or f32 each; the weights are
    [channels], gate, scale and shift [channels] (shared) or [sequences, channels] with ``offsets`` saying
    which rows are whose; all of these have one type, bf16 or f32. Every parameter may be left out.
    With ``training`` forward() keeps what backward() needs (not copies).
    """

    def __init__(self, channels, *, post="none", pre="rms", eps=1e-6, alpha=1.0, training=True):
        _need(post in _KINDS and pre in _KINDS, f"norms are one of {sorted(_KINDS)}")
        self.channels, self.post, self.pre = channels, post, pre
        self.eps, self.alpha, self.training = eps, alpha, training
        self._saved = None

    def _rows(self, t, like, dtype, dev, name):
        """Checks a [.., channels] tensor and gives its row stride (0: contiguous)."""
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
        _need(t.device == dev, f"{name} is on {t.device}, not {dev}")
        _need(t.shape == like.shape, f"{name} must have the shape {tuple(like.shape)}, not {tuple(t.shape)}")
        if t.is_contiguous():
            return 0
        _need(t.stride(-1) == 1, f"{name}: the elements of a row must be consecutive")
        if t.dim() == 2:
            return t.stride(0) if t.shape[0] > 1 else 0
        row = t.stride(1) if t.shape[1] > 1 else t.stride(0)
        _need(t.shape[0] <= 1 or t.shape[1] <= 1 or t.stride(0) == t.shape[1] * t.stride(1),
              f"{name}: the sequences must lie one behind the other")
        _need(row >= self.channels, f"{name}: expanded tensors are not taken")
        return row

    def _params(self, x, y, seqs, rows, params):
        dtypes = {t.dtype for t in params.values() if t is not None}
        _need(len(dtypes) <= 1, "weights, gate, scale and shift must have one type")
        p = P.prism_norm_params(rows=rows, channels=self.channels, seqs=seqs, stream_dtype=P._dtype(x),
                                branch_dtype=P._dtype(x if y is None else y),
                                param_dtype=P._dtype(next(t for t in params.values() if t is not None)) if dtypes else P.PRISM_F32,
                                post_norm=_KINDS[self.post], pre_norm=_KINDS[self.pre], eps=self.eps, alpha=self.alpha)
        for name, t in params.items():
            if t is None:
                continue
            _need(t.device == x.device, f"{name} is on {t.device}, not {x.device}")
            _need(t.shape[-1] == self.channels and (t.dim() == 1 or (t.dim() == 2 and "weight" not in name and t.shape[0] in (1, seqs))),
                  f"{name} has the shape {tuple(t.shape)}")
            _need(t.stride(-1) == 1, f"{name}: the elements of a row must be consecutive")
            if t.dim() == 2 and t.shape[0] > 1:
                _need(t.stride(0) >= self.channels, f"{name}: expanded tensors are not taken; pass [channels]")
                setattr(p, name + "_stride", t.stride(0))
        return p

    def forward(self, x, y=None, *, offsets=None, post_weight=None, gate=None, weight=None, scale=None, shift=None,
                x_out=None, h=None, y_norms=None, h_dtype=None):
        """(x_out, h). Without y: (x, N_pre(x) weight (1 + scale) + shift). ``y_norms`` (float [rows]) receives
        the Euclidean norms of y's rows; ``h_dtype`` is the type of h where there is no y (default: x's)."""
        dev = x.device
        _need(dev.type == "cuda", "block norms run on a CUDA device")
        _need(x.dim() in (2, 3) and x.shape[-1] == self.channels,
              f"x must be [rows, {self.channels}] or [sequences, rows, {self.channels}], not {tuple(x.shape)}")
        mods = [t for t in (gate, scale, shift) if t is not None and t.dim() == 2 and t.shape[0] > 1]
        if offsets is not None:
            _need(x.dim() == 2, "offsets belong to a 2-D x")
            _index(offsets, None, dev, "offsets")
            seqs = offsets.numel() - 1
        else:
            seqs = x.shape[0] if x.dim() == 3 else (mods[0].shape[0] if mods else 1)
        rows = x.shape[0] if x.dim() == 2 else x.shape[0] * x.shape[1]
        if seqs == 0:
            _need(rows == 0 or offsets is not None, "rows without sequences")
        _need(seqs >= 1 or rows == 0, "offsets without sequences")
        seqs = max(seqs, 1)
        params = dict(post_weight=post_weight, gate=gate, weight=weight, scale=scale, shift=shift)
        p = self._params(x, y, seqs, rows, params)
        branch = (h.dtype if h is not None else h_dtype or x.dtype) if y is None else y.dtype
        p.branch_dtype = {torch.bfloat16: P.PRISM_BF16, torch.float32: P.PRISM_F32}.get(branch, -1)
        p.x_row_stride = self._rows(x, x, None, dev, "x")
        with _on_device(dev):
            if y is not None:
                p.y_row_stride = self._rows(y, x, None, dev, "y")
                if x_out is None:
                    x_out = torch.empty(x.shape, dtype=x.dtype, device=dev)
                p.x_out_row_stride = self._rows(x_out, x, x.dtype, dev, "x_out")
            if h is None:
                h = torch.empty(x.shape, dtype=branch, device=dev)
            p.h_row_stride = self._rows(h, x, branch, dev, "h")
            if y_norms is not None:
                _need(y_norms.dtype == torch.float32 and y_norms.is_contiguous() and y_norms.numel() == rows
                      and y_norms.device == dev, f"y_norms must be {rows} contiguous floats on {dev}")
            P.prism_block_norm_fwd(p, x, y, offsets, post_weight, gate, weight, scale, shift,
                                   x_out if y is not None else None, h, y_norms)
        kept = x if y is None else x_out
        if y is None:
            p.x_out_row_stride = p.x_row_stride
        self._saved = (p, kept, y, offsets, params) if self.training else None
        return kept, h

    def backward(self, dh, dx_out=None, dx=None, dy=None):
        """Gradients of the last forward(): a dict of dx, dy and the parameters' (None for what was left out),
        shaped and typed like what they belong to. ``dx_out``: the gradient that reaches the residual stream behind
        the block (None: zero)."""
        _need(self._saved is not None, "backward() needs a forward() with training=True before it")
        p, kept, y, offsets, params = self._saved
        dev = kept.device
        branch = torch.float32 if p.branch_dtype == P.PRISM_F32 else torch.bfloat16
        p.dh_row_stride = self._rows(dh, kept, branch, dev, "dh")
        if dx_out is not None:
            p.dx_out_row_stride = self._rows(dx_out, kept, kept.dtype, dev, "dx_out")
        with _on_device(dev):
            if dx is None:
                dx = torch.empty(kept.shape, dtype=kept.dtype, device=dev)
            p.dx_row_stride = self._rows(dx, kept, kept.dtype, dev, "dx")
            if y is not None:
                if dy is None:
                    dy = torch.empty(y.shape, dtype=y.dtype, device=dev)
                p.dy_row_stride = self._rows(dy, kept, y.dtype, dev, "dy")
            grads = {n: None if t is None or (y is None and n in ("gate", "post_weight")) else
                     torch.empty(t.shape, dtype=t.dtype, device=dev) for n, t in params.items()}
            ws = torch.empty(P.prism_block_norm_workspace_size(p), dtype=torch.uint8, device=dev)
            P.prism_block_norm_bwd(p, kept, y, offsets, params["post_weight"], params["gate"], params["weight"],
                                   params["scale"], dh, dx_out, dx, dy, grads["post_weight"], grads["gate"],
                                   grads["weight"], grads["scale"], grads["shift"], ws)
        return {"dx": dx, "dy": dy, **{"d" + n: g for n, g in grads.items()}}
