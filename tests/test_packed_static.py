"""Static checks of the packed attention kernels' sources (CPU): every mbarrier of the barrier area is
initialised exactly once, no two share a place, and no kernel names a copy with cluster multicast."""

import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "dynamic_block_sparse_variance_b200" / "csrc"
SOURCES = sorted(p.name for p in CSRC.glob("packed_*_tc.cuh"))


def _kernels(text):
    """Texts of the kernels and of the device functions that are a CTA's whole work."""
    starts = [m.start() for m in re.finditer(r"__global__ void|void packed_\w+_cta\(", text)]
    for a, b in zip(starts, starts[1:] + [len(text)]):
        yield text[a:b]


@pytest.mark.parametrize("src", SOURCES)
def test_barriers_are_initialised_once_and_apart(src):
    seen = 0
    for body in _kernels((CSRC / src).read_text()):
        one = dict(re.findall(r"const uint32_t (b_\w+) = sBar(?: \+ 8u \* (\d+))?;", body))
        many = dict(re.findall(r"auto (b_\w+) = \[&\]\(int \w+\) \{ return sBar \+ 8u \* (?:\((\d+) \+ \w+\)|\w+); \};", body))
        if not one and not many:
            continue
        seen += 1
        inits = re.findall(r"mbar_init\((b_\w+)", body)
        assert sorted(inits) == sorted([*one, *many]), src
        starts = sorted([int(v or 0) for v in one.values()] + [int(v or 0) for v in many.values()])
        assert len(set(starts)) == len(starts), f"{src}: two barriers at one place"
    assert seen >= 1


def test_sources_are_found():
    assert SOURCES
    for src in SOURCES:
        assert ".multicast::cluster" not in (CSRC / src).read_text()
