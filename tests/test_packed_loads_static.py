"""Kernels that are launched behind a running one read global memory with coherent loads only: the kernel before
them may write what they read while they are already resident."""

import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "dynamic_block_sparse_variance_b200" / "csrc"
SOURCES = ["block_norm.cuh", "packed_attn.cuh", "packed_bwd_tc.cuh", "packed_common.cuh", "packed_fwd_rows.cuh", "packed_fwd_tc.cuh"]


def _code(name):
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def test_every_kernel_launched_behind_is_in_these_files():
    host = _code("packed_host.cuh")
    names = set(re.findall(r"launch_behind\((\w+_kernel)", host)) | set(re.findall(r"= (\w+_kernel)<", host))
    defined = {n for s in SOURCES for n in re.findall(r"\s(\w+_kernel)\(const", _code(s))}
    assert len(names) >= 9 and names <= defined, names - defined


def test_no_non_coherent_loads():
    for name in SOURCES:
        found = re.findall(r"__ldg|__restrict__|ld\.global\.nc|__ldcs|__ldlu", _code(name))
        assert not found, (name, found)
