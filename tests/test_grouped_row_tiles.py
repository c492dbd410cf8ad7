"""The grouped product's tiles of an expert's rows (csrc/row_tiles.h), on the host: up to the most rows that a call takes, where 32 bits
are nearly full, against Python's integers."""
import ctypes
import os
import random
import subprocess

import pytest

from moe_grouped_gemm_mxfp8_gb300 import build as build_mod

MOST = (1 << 31) - 1024  # rows of a call

CODE = """
#include "row_tiles.h"
extern "C" void row_tile(int rows, int n, int i, int* first, int* count) { gmmfr::row_tile(rows, n, i, *first, *count); }
"""


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_tiles")
    src, lib = d / "row_tiles.cpp", d / "row_tiles.so"
    src.write_text(CODE)
    # -fwrapv: a sum that does not fit in 32 bits comes out wrong, the same way each time
    subprocess.run(["g++", "-O1", "-std=c++17", "-fwrapv", "-fPIC", "-shared", "-I", build_mod.CSRC, str(src), "-o", str(lib)], check=True)
    fn = ctypes.CDLL(os.fspath(lib)).row_tile

    def call(rows, n, i):
        first, count = ctypes.c_int(), ctypes.c_int()
        fn(rows, n, i, ctypes.byref(first), ctypes.byref(count))
        return first.value, count.value

    return call


def _width(rows, n):
    return -(-(-(-rows // n)) // 32) * 32


@pytest.mark.parametrize("rows", list(range(1, 1200)) + [4095, 4096, 4097, 65535, 65536, 65537])
def test_the_tiles_are_the_rows(tile, rows):
    n = -(-rows // 256)
    at = 0
    for i in range(n):
        first, count = tile(rows, n, i)
        assert first == at and 0 < count <= _width(rows, n) <= 256
        at += count
    assert at == rows


def _many():
    rng = random.Random(1)
    # above 2139127680 rows, rows + n is past 2^31
    edge = 2139127680
    return [MOST, MOST - 1, MOST - 255, MOST - 256, edge - 1, edge, edge + 1, edge + 256, edge + 257, 1 << 30, (1 << 30) + 1] \
        + [rng.randint(edge, MOST) for _ in range(200)] + [rng.randint(1, MOST) for _ in range(200)]


@pytest.mark.parametrize("rows", _many())
def test_of_most_rows_too(tile, rows):
    n = -(-rows // 256)
    w = _width(rows, n)
    for i in {0, n // 3, n // 2, n - 2, n - 1} - {-1}:
        assert tile(rows, n, i) == (i * w, min(w, rows - i * w))
        assert tile(rows, n, i)[1] > 0
