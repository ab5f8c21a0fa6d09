"""How the attention kernels deal a line of units to their CTAs, against plain
integers.  The functions are the kernels' own, compiled for the host."""
import ctypes
import random
import shutil
import subprocess
from pathlib import Path

import numpy as np
import pytest

CSRC = Path(__file__).resolve().parents[1] / "kv_cache_compression_cachegen_b200" / "csrc"
SOURCE = """
#include "shares.cuh"
extern "C" void shares(int64_t units, int ctas, int64_t* out) {
  for (int c = 0; c <= ctas; ++c) out[c] = cg::share_of(c, units, ctas);
}
extern "C" void owners(const int64_t* u, int n, int64_t units, int ctas, int* out) {
  for (int i = 0; i < n; ++i) out[i] = cg::cta_of(u[i], units, ctas);
}
extern "C" int most_ctas() { return cg::kMaxRowCtas; }
extern "C" int row_ctas_per_sm() { return cg::kRowCtasPerSm; }
extern "C" int64_t narrow() { return cg::kNarrowUnits; }
// the request that a join finds for row t, and the one of the slot that it takes
extern "C" void agree(const int* q, int B, int tokens, int group, int tile, int t, int member,
                      int* out) {
  const int lo = cg::last_not_above(B, t, cg::FirstRows{q});
  out[0] = lo;
  const cg::FirstSlots slots{q, tokens, group, tile};
  const int x = slots(lo) + ((t - q[lo]) * group + member) / tile;
  out[1] = cg::last_not_above(B, x, slots);
  out[2] = x;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    compiler = shutil.which("g++")
    assert compiler, "g++ is part of the toolchain"
    at = tmp_path_factory.mktemp("shares")
    (at / "shares.cpp").write_text(SOURCE, "utf-8")
    subprocess.run([compiler, "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}",
                    str(at / "shares.cpp"), "-o", str(at / "shares.so")], check=True)
    out = ctypes.CDLL(str(at / "shares.so"))
    out.narrow.restype = ctypes.c_int64
    return out


def check(lib, units, ctas):
    got = np.empty(ctas + 1, np.int64)
    lib.shares(ctypes.c_int64(units), ctas, got.ctypes.data_as(ctypes.c_void_p))
    want = [c * units // ctas for c in range(ctas + 1)]
    assert got.tolist() == want, (units, ctas)
    if units >= ctas:  # no share is empty: the first and last unit of each are its own
        u = np.array([w for c in range(ctas) for w in (want[c], want[c + 1] - 1)], np.int64)
        mine = np.empty(len(u), np.int32)
        lib.owners(u.ctypes.data_as(ctypes.c_void_p), len(u), ctypes.c_int64(units), ctas,
                   mine.ctypes.data_as(ctypes.c_void_p))
        assert mine.tolist() == [c for c in range(ctas) for _ in range(2)], (units, ctas)


def test_every_number_of_ctas_around_the_limits_of_32_bits(lib):
    for ctas in range(1, 321):
        border = -(-(1 << 32) // ctas)  # from here units * ctas passes 32 bits
        for units in (ctas, ctas + 1, 1000003, border - 1, border, border + 1, (1 << 23) - 1,
                      1 << 23, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, 1 << 31, 1 << 40):
            if units >= ctas:
                check(lib, units, ctas)


@pytest.mark.parametrize("ctas", [148, 160, 296, 320])
@pytest.mark.parametrize("units", [14510024, 14510025, 14767304, 16000000, 16777215, 16777216])
def test_the_sizes_of_long_batches(lib, ctas, units):
    check(lib, units, ctas)


def test_the_narrow_arithmetic_fits_the_most_ctas(lib):
    assert lib.narrow() * lib.most_ctas() <= 1 << 32
    assert lib.most_ctas() == 160 * lib.row_ctas_per_sm()


@pytest.mark.parametrize("rising", [True, False])
def test_joins_and_slots_find_the_same_request(lib, rising):
    # lengths out of order are a caller's mistake that must not lead a join astray
    r = random.Random(int(rising))
    out = (ctypes.c_int * 3)()
    for _ in range(3000):
        B, tokens = r.randint(1, 12), r.choice([40, 700, 5000])
        group, tile = r.choice([1, 3, 4, 64]), r.choice([128, 256])
        inside = [r.randint(0, tokens) for _ in range(B + 1)]
        starts = sorted(inside) if rising else [x + r.choice([0, 0, -9000, 9000]) for x in inside]
        q = (ctypes.c_int * (B + 1))(*starts)
        for _ in range(20):
            t, member = r.randrange(tokens), r.randrange(group)
            lib.agree(q, B, tokens, group, tile, t, member, out)
            first, last = starts[out[0]], starts[out[0] + 1]
            if not 0 <= first <= t < last <= tokens:
                continue  # the join leaves this row out
            assert out[0] == out[1], (starts, t)
            assert 0 <= out[2] < tokens * group // tile + B
