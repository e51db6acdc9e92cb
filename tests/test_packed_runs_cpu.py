"""The cut of sequences into runs of rows (csrc/packed_runs.cuh), compiled for the host: the runs cover a sequence
exactly, up to the largest row numbers that the entry points take."""

import ctypes
import pathlib
import re
import subprocess

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "dynamic_block_sparse_variance_b200" / "csrc"
LIMIT = 2 ** 31 - 256      # rows

SOURCE = """
#include "packed_runs.cuh"
extern "C" int rows(int begin, int len, int64_t piece, int unit, int *r) { return prism::run_rows(begin, len, piece, unit, r[0], r[1]); }
extern "C" int count(int len, int unit) { return prism::run_count(len, unit); }
extern "C" int64_t length(int64_t rows, int seqs, int ctas, int64_t least) { return prism::run_length(rows, seqs, ctas, least); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("runs") / "runs.so"
    subprocess.run(["g++", "-O1", "-fwrapv", "-x", "c++", "-shared", "-fPIC", "-I", str(CSRC), "-", "-o", str(out)], input=SOURCE.encode(),
                   check=True)
    so = ctypes.CDLL(str(out))
    so.length.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    so.length.restype = ctypes.c_int64
    so.rows.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    return so


def _run(lib, begin, length, piece, unit):
    r = (ctypes.c_int * 2)()
    return (r[0], r[1]) if lib.rows(begin, length, piece, unit, r) else None


@pytest.mark.parametrize("rows", [1, 147, 61440, 2 ** 30 + 12345, LIMIT])
@pytest.mark.parametrize("seqs", [1, 2, 147, 200])
def test_runs_cover_a_sequence_exactly(lib, rows, seqs):
    """Sequences of one row and a long one last or first; runs as long as a share of the rows or all of them."""
    short = min(seqs - 1, rows - 1)
    for begin, length in ((short, rows - short), (0, rows - short)):
        for unit in {1 if rows < 10 ** 6 else rows // 148, max(1, -(-rows // 148)), max(1, -(-rows // max(1, 148 - seqs))), rows, LIMIT}:
            n = lib.count(length, unit)
            assert n == -(-length // unit)
            at = begin
            for piece in range(n):
                r0, r1 = _run(lib, begin, length, piece, unit)
                assert r0 == at and r0 < r1 <= begin + length and r1 - r0 <= unit
                at = r1
            assert at == begin + length
            assert _run(lib, begin, length, n, unit) is None and _run(lib, begin, length, -1, unit) is None


@pytest.mark.parametrize("ctas", [148, 296, 1184])
@pytest.mark.parametrize("rows", [61440, LIMIT])
def test_the_longest_sequence_is_shared_out(lib, rows, ctas):
    """However many sequences there are, one of half the rows is cut into a third of the CTAs' number of runs at least,
    and with few sequences there are no more runs than CTAs."""
    for seqs in (1, 12, 37, 74, 147, 148, 150, 1000, 65534):
        unit = lib.length(rows, seqs, ctas, 1)
        assert lib.count(rows // 2, unit) >= ctas // 3
        if seqs <= ctas // 4:
            assert rows // unit + seqs <= ctas + 1
    assert lib.length(10, 1, ctas, 16) == 16


def test_no_runs_without_rows(lib):
    assert lib.count(0, 7) == 0 and _run(lib, 5, 0, 0, 7) is None


def test_the_norms_take_their_runs_from_here():
    text = (CSRC / "block_norm.cuh").read_text()
    assert text.count("run_rows(") == 1 and text.count("run_count(") == 1
    assert not re.search(r"\+ a\.unit", text)
