"""Which tensors of a call share memory, as the argument checks see it: against
sets of bytes, for random strided layouts (no GPU needed)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++")
SOURCE = """
#include "la_overlap.cuh"
using namespace la;
static Region make(const long long* t)   // address, element bytes, cols, 3 counts, 3 strides
{
    return region(reinterpret_cast<const void*>(t[0]), (size_t)t[1], t[2], {t[3], t[4], t[5]}, {t[6], t[7], t[8]});
}
extern "C" int pair(const long long* a, const long long* b) { return shared(make(a), make(b)); }
extern "C" int alone(const long long* a) { return overlaps_itself(make(a)); }
"""


@pytest.fixture(scope="module")
def native(tmp_path_factory):
    if CXX is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("overlap")
    (d / "t.cpp").write_text(SOURCE)
    so = str(d / "t.so")
    subprocess.run([CXX, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "causal_kernelized_linear_la_b200", "csrc"), str(d / "t.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def _args(t):
    return (ctypes.c_longlong * 9)(*t)


def _entries(t):
    p, e, cols, counts, strides = t[0], t[1], t[2], t[3:6], t[6:9]
    for i in range(counts[0]):
        for j in range(counts[1]):
            for k in range(counts[2]):
                at = p + (i * strides[0] + j * strides[1] + k * strides[2]) * e
                yield (i, j, k), range(at, at + cols * e)


def _bytes(t):
    return {x for _, r in _entries(t) for x in r}


def _overlaps_itself(t):
    """Entries that differ in an axis that moves (an axis of stride 0 shows the same bytes again)."""
    seen = {}
    for idx, r in _entries(t):
        idx = tuple(i if s else 0 for i, s in zip(idx, t[6:9]))
        for x in r:
            if seen.setdefault(x, idx) != idx:
                return True
    return False


def _random(rng):
    e, cols = rng.choice((2, 4)), rng.randint(1, 5)
    counts = [rng.choice((1, 1, 2, 3, 4)) for _ in range(3)]
    if rng.random() < 0.6:         # nested, perhaps with gaps, in any order of axes
        order, step, strides = rng.sample(range(3), 3), cols, [0, 0, 0]
        for k in order:
            step += rng.choice((0, 0, 1, 3, 7))
            strides[k] = step
            step *= counts[k]
        if rng.random() < 0.2:
            strides[rng.randrange(3)] = 0
    else:
        strides = [rng.randint(0, 20) for _ in range(3)]
    return [1000 + e * rng.randint(0, 60), e, cols, *counts, *strides]


def test_random_layouts(native):
    rng, hits = random.Random(5), 0
    for _ in range(4000):
        a = _random(rng)
        b = _random(rng)
        if rng.random() < 0.4:     # two parts of one buffer
            b = [a[0] + a[1] * rng.randint(0, 12), a[1], rng.randint(1, 4), *a[3:]]
        want = bool(_bytes(a) & _bytes(b))
        hits += want
        assert bool(native.pair(_args(a), _args(b))) == want == bool(native.pair(_args(b), _args(a))), (a, b)
        assert bool(native.alone(_args(a))) == _overlaps_itself(a), a
    assert 800 < hits < 3200


def test_large_layouts(native):
    """Sizes of real calls, where no list of bytes can be made."""
    B, N, H, d = 64, 1 << 20, 40, 128
    row = H * d
    part = lambda first, heads: [(1 << 40) + 2 * first * d, 2, d, B, heads, N, N * row, d, row]  # noqa: E731
    q, k, v = part(0, 32), part(32, 4), part(36, 4)
    assert not native.pair(_args(q), _args(k)) and not native.pair(_args(k), _args(v)) and not native.pair(_args(v), _args(q))
    assert native.pair(_args(part(0, 33)), _args(k)) and native.pair(_args(part(35, 2)), _args(k))
    assert not native.alone(_args(q))
    gap = [(1 << 40) + 2 * (N * row * 3 - d), 2, d, 1, 1, 1, 0, 0, 0]         # the last row of batch 2's last column
    assert native.pair(_args(gap), _args(v)) and not native.pair(_args(gap), _args(k))
    # rows of unlike strides: they meet somewhere, and the search ends
    a, b = [1 << 40, 2, 64, 1, 1, N, 0, 0, 100], [1 << 40, 2, 64, 1, 1, N, 0, 0, 9973]
    assert native.pair(_args(a), _args(b))
    empty = [1 << 40, 2, 64, 1, 0, N, 0, 0, 100]
    assert not native.pair(_args(empty), _args(a)) and not native.pair(_args([0] + a[1:]), _args(a))
