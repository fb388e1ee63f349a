"""The search for a bound among logits (csrc/bound.h), compiled for the host.

Keys order finite logits as whole numbers.  What the search returns must be reached by as many threads as asked
for, and by at most a quarter and one more unless the next key is not; 0 only where fewer have a finite logit; whatever the logits'
sign and size, in a bounded number of counts.
"""
import ctypes
import os
import random
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_long_gb300", "csrc")
SOURCE = """
#include "bound.h"
extern "C" uint32_t search(int need, uint32_t top, uint32_t lo, const uint32_t* best, int threads, int limit, int* counts) {
  *counts = 0;
  struct Endless {};
  try {
    return dsa::sample::reached_by(need, top, lo, [&](uint32_t key) {
      if (++*counts > limit) throw Endless();
      int n = 0;
      for (int i = 0; i < threads; ++i) n += best[i] >= key;
      return n;
    });
  } catch (Endless) { return 1; }
}
"""
LIMIT, THREADS, INF = 60, 256, float("inf")      # 10 counts to a first bound, 8 halves of the larger end, 32 of the keys


def key(x):
    u = struct.unpack("<I", struct.pack("<f", x + 0.0))[0]
    return ~u & 0xFFFFFFFF if u >> 31 else u | 0x80000000


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("bound")
    (d / "s.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "s.cpp"), "-o", str(d / "s.so")], check=True)
    f = ctypes.CDLL(str(d / "s.so")).search
    f.restype, f.argtypes = ctypes.c_uint32, [ctypes.c_int, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_int,
                                              ctypes.c_int, ctypes.c_void_p]

    def run(need, best, top=None, lo=0):
        keys = (ctypes.c_uint32 * len(best))(*[key(x) for x in best])
        counts = ctypes.c_int()
        r = f(need, key(max(best)) if top is None else top, lo, keys, len(best), LIMIT, ctypes.byref(counts))
        assert counts.value <= LIMIT
        return r, counts.value

    return run


def check(search, need, best, **kw):
    bound, counts = search(need, best, **kw)
    keys = [key(x) for x in best]
    reach = lambda k: sum(b >= k for b in keys)
    if reach(key(-3.4028234663852886e38)) < need:
        assert bound == 0
    else:
        assert bound > 0 and reach(bound) >= need
        assert need == 1 or reach(bound) <= need + need // 4 + 1 or reach(bound + 1) < need
    return counts


@pytest.mark.parametrize("shift", [0, 8, -4, -6, -8, -10, -15, -100, 100, 1000, -1e4, 1e30, -1e30])
def test_logits_of_any_mean(search, shift):
    rng = random.Random(7)
    f32 = lambda x: struct.unpack("<f", struct.pack("<f", x))[0]
    most = 0
    for spread in (0.05, 1.0, 2.5, 8.0):
        for need in (2, 7, 50, 192, 256):
            # the largest of 16 logits, and a few that are likelier
            best = [f32(shift + spread * (max(rng.gauss(0, 1) for _ in range(16)) + (rng.random() < 0.03) * (4 + rng.expovariate(1))))
                    for _ in range(THREADS)]
            most = max(most, check(search, need, best))
    assert most <= LIMIT


def test_any_keys(search):
    rng = random.Random(3)
    lowest = 3.4028234663852886e38
    ends = [-lowest, -1e30, -1e4, -3.0, -1.0, -1e-3, -1e-30, -0.0, 0.0, 1e-45, 1e-30, 0.5, 1.0, 2.0, 1e4, lowest]
    for _ in range(4000):
        a, b = sorted(rng.choice(ends) for _ in range(2))
        pick = lambda: rng.choice([a, b]) if b - a > lowest else rng.uniform(a, b)
        best = [struct.unpack("<f", struct.pack("<f", min(max(pick(), -lowest), lowest)))[0] for _ in range(THREADS)]
        for i in range(rng.choice([0, 0, 3, 200, 256])):
            best[i] = -INF
        need = rng.choice([1, 2, 5, 40, 100, 192, 256])
        if best.count(-INF) < THREADS or need > 1:
            check(search, need, best)
        # on from a bound that held before these were seen: the largest known, or any number above it
        s = sorted((key(x) for x in best), reverse=True)
        if need > 1 and s[need - 1] >= 0x00800000:
            lo = rng.choice([0x00800000, s[need - 1], max(0x00800000, s[need - 1] - rng.randrange(1 << 20))])
            check(search, need, best, lo=lo, top=rng.choice([s[0], 0xFFFFFFF0]))


def test_more_threads_than_there_are(search):
    assert search(257, [1.0] * THREADS)[0] == 0 and search(1000, [-5.0] * 100 + [-INF] * 156)[0] == 0
    assert search(3, [2.0, 1.0] + [-INF] * 254)[0] == 0 and 0 < search(2, [2.0, -1e30] + [-INF] * 254)[0] <= key(-1e30)
    assert search(2, [-INF] * THREADS)[0] == 0
