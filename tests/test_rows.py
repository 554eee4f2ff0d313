"""CPU: the host checks for shared bytes of strided tensors (csrc/rows.h),
compiled alone, against sets of bytes."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_gemm_packed_amd", "csrc")
CODE = """
#include "rows.h"
extern "C" int both(const long long* a, const long long* b) {
  return (int)hum::overlap({a[0], a[1], a[2], a[3], a[4], a[5]}, {b[0], b[1], b[2], b[3], b[4], b[5]});
}
extern "C" int self(const long long* a) { return hum::overlaps_itself({a[0], a[1], a[2], a[3], a[4], a[5]}); }
"""


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cpp").write_text(CODE)
    so = d / "rows.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "rows.cpp"), "-o", str(so)],
                   check=True)
    lib = ctypes.CDLL(str(so))
    arr = lambda r: (ctypes.c_longlong * 6)(*r)  # noqa: E731
    return (lambda a, b: lib.both(arr(a), arr(b))), (lambda a: lib.self(arr(a)))


def _bytes(r):
    at, t, h, ts, hs, row = r
    return [at + i * ts + j * hs + k for i in range(t) for j in range(h) for k in range(row)]


def test_against_sets_of_bytes(rows):
    both, self = rows
    g = np.random.default_rng(0)
    seen = {0: 0, 1: 0}
    for n in range(20000):
        def tensor():
            ts, hs = (int(x) for x in g.integers(-40, 41, 2))
            return [int(g.integers(1000, 1080)), int(g.integers(0, 6)), int(g.integers(0, 6)), ts, hs, int(g.integers(1, 9))]
        a, b = tensor(), tensor()
        if n % 3 == 0:
            b[3:5] = a[3:5]
        elif n % 3 == 1:
            b[3] = a[3]
        x, y = _bytes(a), _bytes(b)
        want = bool(set(x) & set(y))
        assert both(a, b) == both(b, a) == int(want), (a, b)
        assert bool(self(a)) == (len(set(x)) < len(x)), a
        seen[int(want)] += 1
    assert min(seen.values()) > 2000


def test_slices_of_a_fused_product(rows):
    """q, k and v side by side in every token, by heads in turn, or head by head; 2^24 tokens cost no more than four."""
    both, self = rows
    for t in (4, (1 << 24) - 1):
        f = 48 * 256                                        # bytes of a token: 32 + 8 + 8 heads of 128 bf16
        q, k, v = ([1 << 20, t, 32, f, 256, 256], [(1 << 20) + 32 * 256, t, 8, f, 256, 256],
                   [(1 << 20) + 40 * 256, t, 8, f, 256, 256])
        assert not any(both(a, b) for a, b in ((q, k), (q, v), (k, v))) and not self(q)
        wide = q[:2] + [33] + q[3:]
        assert both(wide, k) and not both(wide, v)
        even, odd = [1 << 20, t, 24, f, 512, 256], [(1 << 20) + 256, t, 24, f, 512, 256]
        assert not both(even, odd) and both(even, [(1 << 20) + 255] + odd[1:]) and not self(even)
        turned, more = [1 << 20, t, 8, 256, t * 256, 256], [(1 << 20) + 8 * t * 256, t, 8, 256, t * 256, 256]
        assert not both(turned, more) and both(turned, [more[0] - 256] + more[1:]) and not self(turned)
        assert both(q, [q[0] + 256] + q[1:]) and both(q, [q[0] + f] + q[1:])
        assert self([1 << 20, t, 8, 256, 256, 256]) and self([0, t, 1, 0, 0, 2]) and not self([0, 1, 1, 0, 0, 2])
    assert self([0, 3, 1, 511, 0, 512]) and not self([0, 3, 1, -512, 0, 512])
    # strides past anything that memory holds
    assert not self([0, 1 << 23, 4096, 1 << 62, 1 << 49, 256])
    # too many rows with different strides, one inside the other
    assert both([0, 1 << 23, 2, 1024, 256, 256], [512, 1 << 23, 2, 1025, 256, 256]) == 2
