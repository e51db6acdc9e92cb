"""Forms of the block norms beside the usual one: many sequences of very different lengths, the norm behind a block
alone (no h), and a backward without a gradient of h. Bounds as in tests/test_gpu_block_norm.py."""

import numpy as np
import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.packed import BlockNorm
from tests import packed_reference as ref
from tests import test_gpu_block_norm as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs", [17, 74, 150, 1000])
@pytest.mark.parametrize("mods", ["per", "shared"])
@pytest.mark.parametrize("stream,branch,param,c", [("bf16", "bf16", "f32", 128), ("f32", "bf16", "bf16", 1536)])
def test_many_sequences(stream, branch, param, c, mods, seqs):
    """One sequence with half of the rows, empty ones, and short ones; more sequences than a wave has CTAs."""
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 5, seqs)
    lens[seqs // 2] = 1000
    off = ref.offsets(lens)
    a = base._inputs(off[-1], c, seqs, stream, branch, param, mods, seed=seqs)
    norm = BlockNorm(c, post="rms", pre="layer", alpha=0.7)
    x_out, h = norm.forward(a["x"], a["y"], offsets=base._ints(off), **{n: a[n] for n in base.NAMES})
    g = norm.backward(a["dh"], a["dx_out"])
    P.prism_device_status()
    want = base._reference(a, off, "rms", "layer", 0.7, kept=base._f64(x_out))
    base._within(x_out, want["x_out"], base._tol(want["x_out"], x_out.dtype, 4.0), "x_out")
    base._within(h, want["h"], base._tol(want["h"], h.dtype, 8.0), "h")
    base._check_grads(g, a, want, 0.7, f"{seqs} sequences")


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("stream,branch,c", [("bf16", "bf16", 256), ("f32", "bf16", 4104), ("bf16", "f32", 712)])
def test_behind_a_block_alone(stream, branch, c, post):
    """h NULL: x_out and the norms of y, with the bits of the whole form."""
    off = ref.offsets([20, 0, 31])
    a = base._inputs(51, c, 3, stream, branch, "f32", "per", seed=c)
    off_d = base._ints(off)
    norm = BlockNorm(c, post=post, pre="rms", alpha=0.6)
    yn, alone_yn = (torch.empty(51, device="cuda") for _ in range(2))
    x_out, _ = norm.forward(a["x"], a["y"], offsets=off_d, post_weight=a["post_weight"], gate=a["gate"], y_norms=yn)
    types = {"bf16": P.PRISM_BF16, "f32": P.PRISM_F32}
    p = P.prism_norm_params(rows=51, channels=c, seqs=3, stream_dtype=types[stream], branch_dtype=types[branch], param_dtype=P.PRISM_F32,
                            post_norm=("none", "rms", "layer").index(post), pre_norm=P.PRISM_NORM_RMS, eps=1e-6, alpha=0.6, gate_stride=c)
    alone = torch.empty_like(x_out)
    P.prism_block_norm_fwd(p, a["x"], a["y"], off_d, a["post_weight"], a["gate"], None, None, None, alone, None, alone_yn)
    P.prism_device_status()
    assert torch.equal(alone, x_out) and torch.equal(alone_yn, yn)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("stream,branch,c", [("bf16", "bf16", 256), ("f32", "bf16", 4104), ("bf16", "f32", 712)])
def test_backward_without_a_gradient_of_h(stream, branch, c, post):
    """Only what reaches the residual stream: what a zero dh gives."""
    off = ref.offsets([20, 0, 31])
    a = base._inputs(51, c, 3, stream, branch, "f32", "per", seed=c + 1)
    norm = BlockNorm(c, post=post, pre="layer", alpha=0.6)
    x_out, _ = norm.forward(a["x"], a["y"], offsets=base._ints(off), **{n: a[n] for n in base.NAMES})
    g = norm.backward(None, a["dx_out"])
    P.prism_device_status()
    zero = dict(a, dh=torch.zeros_like(a["dh"]))
    want = base._reference(zero, off, post, "layer", 0.6, kept=base._f64(x_out))
    base._check_grads(g, zero, want, 0.6, post)
    assert all((g[n] == 0).all() for n in ("dweight", "dscale", "dshift"))
    with pytest.raises(P.PrismError):
        norm.backward(None)
