"""Whether two parts of memory meet (csrc/kda_span.h), against sets of bytes (no GPU needed)."""
import ctypes
import os
import random
import subprocess

import pytest

from recompute_kda_chunkwise_gb300 import build as kbuild

SOURCE = """
#include "kda_span.h"
extern "C" int span_meet(uint64_t a, int64_t an, uint64_t b, int64_t rows, int64_t bytes, int64_t step) {
  return kda::meet(kda::whole("a", reinterpret_cast<void*>(a), an), {"b", b, rows, bytes, step});
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    d = tmp_path_factory.mktemp("span")
    (d / "span.cpp").write_text(SOURCE)
    csrc = os.path.join(os.path.dirname(kbuild.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-I", csrc, str(d / "span.cpp"), "-o",
                    str(d / "span.so")], check=True)
    fn = ctypes.CDLL(str(d / "span.so")).span_meet
    fn.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    return fn


def test_against_sets_of_bytes(meet):
    rng = random.Random(0)
    hits = 0
    for _ in range(20_000):
        a, an, b = rng.randrange(1, 60), rng.randrange(0, 12), rng.randrange(1, 60)
        rows, n = rng.randrange(0, 5), rng.randrange(0, 7)
        step = n + rng.randrange(0, 9) or 1
        want = set(range(a, a + an)) & {b + i * step + e for i in range(rows) for e in range(n)}
        assert meet(a, an, b, rows, n, step) == bool(want), (a, an, b, rows, n, step)
        hits += bool(want)
    assert 2000 < hits < 18_000


def test_far_addresses_and_long_steps(meet):
    base, big = 0x7F00_0000_0000, 1 << 38
    assert meet(base + 5 * big, 16, base, 6, 16, big) == 1
    assert meet(base + 5 * big + 16, 16, base, 6, 16, big) == 0
    assert meet(base + 6 * big, 16, base, 6, 16, big) == 0
    assert meet(base - 16, 16, base, 6, 16, big) == 0 and meet(base - 15, 16, base, 6, 16, big) == 1
