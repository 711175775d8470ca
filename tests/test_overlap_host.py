"""The host's check for tensors that share memory (csrc/overlap.h) against the bytes themselves."""
import ctypes
import os
import random
import subprocess

import pytest

from token_level_sparse_pddp_b200 import build as tlsp_build

SOURCE = """
#include "overlap.h"
using namespace tlsp;
static Span span(const long* t) {  // address, run, three axes (n, step)
  Span s((const void*)t[0], t[1]);
  for (int i = 0; i < 3; ++i) s.with(t[2 + 2 * i], t[3 + 2 * i]);
  return s;
}
extern "C" int apart_of(const long* a, const long* b) { return apart(span(a), span(b)); }
extern "C" int distinct_of(const long* a) { return span(a).distinct(); }
"""


@pytest.fixture(scope="module")
def C(tmp_path_factory):
    at = tmp_path_factory.mktemp("overlap")
    src, so = at / "overlap.cpp", at / "overlap.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(tlsp_build.CSRC), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def call(f, *tensors):
        return bool(f(*[(ctypes.c_long * 8)(t[0], t[1], *[x for a in t[2] for x in a],
                                            *([1, 0] * (3 - len(t[2])))) for t in tensors]))
    return type("C", (), {"apart": lambda a, b: call(lib.apart_of, a, b),
                          "distinct": lambda a: call(lib.distinct_of, a)})


def elements(t):
    """Start of each run of bytes."""
    starts = [t[0]]
    for n, step in t[2]:
        starts = [s + i * step for s in starts for i in range(n)]
    return starts


def bytes_of(t):
    return {s + i for s in elements(t) for i in range(t[1])}


def is_distinct(t):
    return len(bytes_of(t)) == len(elements(t)) * t[1]


def test_random_tensors(C):
    """Never apart where a byte is shared; never distinct where two elements share one."""
    r = random.Random(1)
    shared = known = 0
    for _ in range(20000):
        def tensor():
            return (r.randint(100, 300), r.choice([1, 2, 4, 8]),
                    [(r.choice([1, 2, 3, 5]), r.choice([-16, 0, 1, 2, 4, 8, 8, 16, 16, 24, 48, 96]))
                     for _ in range(r.randint(0, 3))])
        a, b = tensor(), tensor()
        common = bool(bytes_of(a) & bytes_of(b))
        said = C.apart(a, b)
        assert not (common and said), (a, b)
        shared += common
        known += said and not common
        assert not C.distinct(a) or is_distinct(a), a
    assert shared > 2000 and known > 4000


def test_slices_of_one_tensor(C):
    """Slices of a wider tensor along any axis, in any order of the axes, are judged exactly."""
    r = random.Random(2)
    both = {True: 0, False: 0}
    for _ in range(4000):
        sizes = [r.randint(1, 6) for _ in range(3)]
        d = r.choice([2, 8])
        order = r.sample(range(3), 3)
        steps, at = [0] * 3, d
        for axis in order:
            steps[axis], at = at, at * sizes[axis]
        cut = r.randrange(3)

        def part():
            lo = [0] * 3
            n = list(sizes)
            lo[cut] = r.randint(0, sizes[cut] - 1)
            n[cut] = r.randint(1, sizes[cut] - lo[cut])
            return (1000 + sum(x * s for x, s in zip(lo, steps)), d, list(zip(n, steps)))
        a, b = part(), part()
        common = bool(bytes_of(a) & bytes_of(b))
        assert C.apart(a, b) == (not common), (a, b)
        assert C.distinct(a) and C.apart(a, (1000 + at, d, [(9, d)]))
        both[common] += 1
    assert min(both.values()) > 500


def test_halves_of_channels_and_no_elements(C):
    wide = 1 << 40
    q = (wide, 256, [(32760, 12 * 512), (12, 512)])
    o = (wide + 256, 256, [(32760, 12 * 512), (12, 512)])
    assert C.apart(q, o) and C.apart(o, q) and not C.apart(q, q)
    assert not C.apart(q, (wide + 254, 256, q[2]))
    assert C.apart(q, (wide, 256, [(0, 512)])) and C.apart((wide, 0, []), q)
    far = [(2 ** 31, 2 ** 62)] * 3                    # more than 64 bits reach
    assert not C.apart((wide, 2, far), (wide, 2, far)) and C.apart((wide, 2, far), (wide - 64, 64, []))
    # gives up on what has no common step, and says shared
    assert not C.apart((0, 2, [(100000, 6)]), (1, 1, [(100000, 4)]))
