"""Arithmetic that filtered sampling decides its borders with (the header the kernels
use, compiled for the CPU)."""
import ctypes
import os
import random
import subprocess
from fractions import Fraction
from math import ceil, floor

import numpy as np
import pytest

from beam_search_top_amd import rtopk

CSRC = os.path.join(os.path.dirname(rtopk.__file__), "csrc")


@pytest.fixture(scope="module")
def arith(tmp_path_factory):
    d = tmp_path_factory.mktemp("filter")
    src = d / "filter.cpp"
    src.write_text('''#define RTOPK_ARITHMETIC_ONLY
#include "rtopk_filter.h"
#include <string.h>
using namespace rtopk;
extern "C" unsigned long long part_(float f, unsigned long long t, int up) { uint32_t b; memcpy(&b, &f, 4); return part_of(b, t, up); }
extern "C" int chunks_(int R, int V, int counts) { return filter_chunks(R, V, counts); }
extern "C" int frac_(int V) { return filter_frac(V); }
''')
    so = d / "filter.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.part_.argtypes = [ctypes.c_float, ctypes.c_ulonglong, ctypes.c_int]
    L.part_.restype = ctypes.c_ulonglong
    return L


def test_parts_of_a_sum_are_exact(arith):
    rng = random.Random(1)
    fs = [0.0, 2.0 ** -149, 3 * 2.0 ** -149, 2.0 ** -126, 2.0 ** -127, 2.0 ** -100, 2.0 ** -64, 2.0 ** -40, 2.0 ** -32, 2.0 ** -31, 2.0 ** -9, 2.0 ** -8, 2.0 ** -7,
          0.5, 0.25, 0.9, 0.95, 1 - 2.0 ** -24, 0.1, 2.0 ** -118, 2.0 ** -117, 2.0 ** -86, 2.0 ** -87]
    fs += [rng.random() for _ in range(400)] + [2.0 ** rng.uniform(-149, 0) * 0.999 for _ in range(400)]
    totals = [1, 2, 3, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 50, 2 ** 53 + 1, 2 ** 62 - 1, 2 ** 62, 2 ** 61 + 1]
    coarse = 0  # products that 53 bits get wrong
    for f in np.float32(fs):
        f = float(f)
        for t in totals + [rng.getrandbits(rng.randint(1, 62)) + 1 for _ in range(12)]:
            t = min(t, 2 ** 62)
            x = Fraction(f) * t
            assert arith.part_(f, t, 0) == floor(x) and arith.part_(f, t, 1) == ceil(x), (f, t)
            coarse += ceil(f * float(t)) != ceil(x)
    assert coarse > 100


def test_weights_of_a_row_sum_below_two_to_the_62(arith):
    for V in (1, 2, 4096, 4097, 250000, 2 ** 24 - 1, 2 ** 24):
        assert V << arith.frac_(V) <= 2 ** 62


def test_where_rows_are_cut(arith):
    # a workspace has room for the call whatever its filters; chunks fill the GPU and are not idle
    for R in list(range(1, 300)) + [512, 4096, 2 ** 20]:
        need = rtopk.rtopk_sample_filtered_workspace_bytes
        for V in (1, 4096, 28671, 28672, 33791, 33792, 40000, 65535, 65536, 100000, 163840, 250000, 2 ** 24):
            c, k = arith.chunks_(R, V, 0), arith.chunks_(R, V, 1)
            assert k in (1, c) and 1 <= c <= 64 and (c == 1 or (R * c <= 512 and V // c >= 4096))
            assert need(R, V) == (need(R, 1) if c == 1 else need(R, 1) + R * 49920)
    # rows of 100000 and more are cut up to where three chunks of each fill the GPU
    assert [arith.chunks_(R, 100000, 0) for R in (1, 8, 128, 129, 170, 171, 256)] == [24, 24, 4, 3, 3, 1, 1]
    assert [arith.chunks_(R, 65535, 0) for R in (128, 129)] == [4, 1]
    assert [arith.chunks_(R, 100000, 1) for R in (1, 65, 66, 129)] == [24, 7, 1, 1]
