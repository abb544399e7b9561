"""The host checks of strided tensors (csrc/op_checks.h) against sets of addresses, on small
tensors: compiled by the host compiler, no GPU."""
import itertools
import os
import random
import subprocess

import pytest

SRC = r"""
#include "op_checks.h"
using ttt::RowTensor;
extern "C" int writable(long p, int e, long w, const long* n, const long* s) {
  return RowTensor((void*)p, e, w, n[0], s[0], n[1], s[1], n[2], s[2]).writable();
}
extern "C" int share(long p, int e, long w, const long* n, const long* s, long p2, long w2, const long* n2, const long* s2) {
  return may_share(RowTensor((void*)p, e, w, n[0], s[0], n[1], s[1], n[2], s[2]),
                   RowTensor((void*)p2, e, w2, n2[0], s2[0], n2[1], s2[1], n2[2], s2[2]));
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory, repo_root):
    import ctypes
    d = tmp_path_factory.mktemp("op_checks")
    (d / "t.cpp").write_text(SRC)
    csrc = os.path.join(repo_root, "weight_sequence_mixing_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", csrc, str(d / "t.cpp"), "-o", str(d / "t.so")], check=True)
    lib = ctypes.CDLL(str(d / "t.so"))
    arr = ctypes.c_long * 3
    lib.w = lambda p, e, w, n, s: bool(lib.writable(ctypes.c_long(p), e, ctypes.c_long(w), arr(*n), arr(*s)))
    lib.s = lambda p, e, a, p2, b: bool(lib.share(ctypes.c_long(p), e, ctypes.c_long(a[0]), arr(*a[1]), arr(*a[2]),
                                                  ctypes.c_long(p2), ctypes.c_long(b[0]), arr(*b[1]), arr(*b[2])))
    return lib


def _places(p, e, w, n, s):
    return [p + e * (sum(i * k for i, k in zip(at, s)) + c) for at in itertools.product(*map(range, n)) for c in range(w)]


def test_a_tensor_that_is_called_writable_never_has_two_elements_in_one_place(lib):
    rng, seen = random.Random(1), [0, 0]
    for _ in range(4000):
        n = [rng.randint(1, 4) for _ in range(3)]
        s = [rng.choice([0, 1, 2, 3, 4, 6, 8, 12, 16, 24, 48]) for _ in range(3)]
        w = rng.randint(1, 4)
        places = _places(4096, 4, w, n, s)
        ok = lib.w(4096, 4, w, n, s)
        seen[ok] += 1
        assert not ok or len(set(places)) == len(places), (n, s, w)
    assert min(seen) > 300


def test_nested_layouts_are_writable(lib):
    for order in itertools.permutations(range(3)):  # contiguous in any order of the dimensions
        n, s, step = (3, 4, 5), [0, 0, 0], 6
        for i in order:
            s[i] = step
            step *= n[i]
        assert lib.w(4096, 2, 6, n, s), (order, s)
    assert lib.w(4096, 2, 6, (1, 1, 5), (0, 0, 6))  # strides of single dimensions do not matter
    assert not lib.w(4096, 2, 6, (2, 1, 5), (0, 0, 6))
    assert not lib.w(4097, 2, 6, (1, 1, 5), (0, 0, 6))


def test_tensors_called_apart_share_no_element(lib):
    rng, apart, exact = random.Random(2), 0, 0
    for _ in range(6000):
        n = [rng.randint(1, 3) for _ in range(3)]
        w = rng.randint(1, 4)
        step = rng.choice([4, 8, 12])
        s = [step * rng.choice([1, 2, 6, 12]) for _ in range(3)]
        other = (w, n, s) if rng.random() < 0.6 else (rng.randint(1, 4), n, [rng.choice([4, 8, 24]) for _ in range(3)])
        p2 = 4096 + rng.randint(-40, 400) * 2
        share = lib.s(4096, 4, (w, n, s), p2, other)
        a, b = set(_places(4096, 4, w, n, s)), set(_places(p2, 4, *other))
        spread = {x + i for x in a for i in range(4)} & {x + i for x in b for i in range(4)}
        apart += not share
        assert share or not spread, (n, s, w, p2, other)
        exact += (not share) and max(a) > min(b) and max(b) > min(a)
    assert apart > 1000 and exact > 100  # columns of one buffer among them


def test_columns_of_one_buffer_are_apart(lib):
    n, s = (2, 1, 700), (700 * 192, 0, 192)
    for k, share in ((126, True), (127, True), (128, False), (129, False), (192, False), (193, True),
                     (64, True)):
        # the first tensor: columns 64..127 of 192; the second: 64 columns from column k on, those past
        # the last being the next token's first
        assert lib.s(1 << 20, 2, (64, n, s), (1 << 20) + 2 * (k - 64), (64, n, s)) == share, k


@pytest.mark.parametrize("n,s,row", [((1, 3, 40), (0, 8, 96), 24),          # [B, N, 4 H d]: heads one behind the other
                                     ((1, 40, 3), (7, 96, 8), 24),      # the same, dimensions in another order
                                     ((2, 3, 20), (20 * 96, 8, 96), 24),    # batch entries one behind the other
                                     ((4, 3, 5), (24, 8, 480), 96)])        # two dense dimensions
def test_column_ranges_of_several_heads_are_apart(lib, n, s, row):
    """The heads of one token lie densely in a wider row: what counts is the whole range of columns."""
    at = 1 << 20
    a = set(_places(at, 2, 8, n, s))
    told = [lib.s(at, 2, (8, n, s), at + 2 * k, (8, n, s)) for k in range(-130, 131)]
    assert told == [bool(a & set(_places(at + 2 * k, 2, 8, n, s))) for k in range(-130, 131)]
    step = max(s)
    for k, share in ((row, False), (row - 1, True), (step - row, False), (step - row + 1, True)):
        assert lib.s(at, 2, (8, n, s), at + 2 * k, (8, n, s)) == share, k
