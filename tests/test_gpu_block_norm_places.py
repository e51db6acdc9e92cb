"""Outputs of the block norms in the place of what backward() starts from: refused, or the last backward()."""

import pytest
import torch

from dynamic_block_sparse_variance_b200 import prism as P
from dynamic_block_sparse_variance_b200.packed import BlockNorm

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _xy(seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(50, 128, generator=gen).to(BF16).cuda() for _ in range(4)]


def test_refused_in_training():
    x, y, *_ = _xy()
    x0, y0 = x.clone(), y.clone()
    norm = BlockNorm(128, post="rms")
    for args, kw in (((x,), dict(h=x)), ((x, y), dict(x_out=y)), ((x, y), dict(h=y)), ((x, y), dict(x_out=y, h=x))):
        with pytest.raises(P.PrismError) as e:
            norm.forward(*args, **kw)
        assert e.value.code == P.PRISM_EINVAL
    assert torch.equal(x, x0) and torch.equal(y, y0)


def test_without_training_any_input_may_be_overwritten():
    x, y, *_ = _xy(1)
    norm = BlockNorm(128, post="rms", training=False)
    before = norm.forward(x)[1]
    x_out, h = norm.forward(x, y)
    a = x.clone()
    assert norm.forward(a, h=a)[1] is a and torch.equal(a, before)
    a, b = x.clone(), y.clone()
    norm.forward(a, b, x_out=b, h=a)
    P.prism_device_status()
    assert torch.equal(b, x_out) and torch.equal(a, h)


@pytest.mark.parametrize("spent", ["dx on x_out", "dy on y", "dx on y", "dy on x_out"])
def test_a_backward_over_what_it_starts_from_is_the_last(spent):
    x, y, dh, dxo = _xy(2)
    norm = BlockNorm(128, post="rms", pre="layer", alpha=0.8)
    x_out, _ = norm.forward(x, y)
    want = norm.backward(dh, dxo)
    again = norm.backward(dh, dxo)
    assert all(torch.equal(want[n], again[n]) for n in ("dx", "dy"))
    out, at = spent.split(" on ")
    got = norm.backward(dh, dxo, **{out: x_out if at == "x_out" else y})
    P.prism_device_status()
    assert all(torch.equal(want[n], got[n]) for n in ("dx", "dy"))
    with pytest.raises(P.PrismError):
        norm.backward(dh, dxo)
