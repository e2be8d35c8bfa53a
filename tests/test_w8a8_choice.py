"""The tile kernel's choice of tiles (csrc/w8a8_choice.h, host code), built here with the host's
compiler: every launch that a call is split into is one that a grid takes, so that a call is
refused before anything runs or not at all, and every size of tile has calls that take it."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "int4_weight_only_03_amd", "csrc")
SHIM = """
#include "w8a8_choice.h"
using namespace w4a16;
extern "C" {
int sizes(int exact) { return exact ? int(std::size(kExactChoices)) : int(std::size(kChoices)); }
int choice(int exact, long R, long E, long N, long K, long part) {
  const TileCall p = {R, E, N, K, E > 0};
  return exact ? least(kExactChoices, p, part).choice : least(kChoices, p, part).choice;
}
long before(int exact, long R, long E, long N, long K) {
  const TileCall p = {R, E, N, K, E > 0};
  return exact ? rows_before_rest(kExactChoices, p) : rows_before_rest(kChoices, p);
}
// workgroups of choice i for `part` rows, threads of all of them
long tiles(int exact, int i, long R, long E, long N, long part) {
  const Choice &c = exact ? kExactChoices[i] : kChoices[i];
  return tiles_of(c.slots, c.rows, TileCall{R, E, N, 128, E > 0}, part);
}
long threads(int exact, int i, long R, long E, long N, long part) {
  const Choice &c = exact ? kExactChoices[i] : kChoices[i];
  return (tiles(exact, i, R, E, N, part) + 7) / 8 * 8 * 64 * c.waves;
}
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    d = tmp_path_factory.mktemp("choice")
    (d / "shim.cpp").write_text("#include <iterator>\n" + SHIM)
    so = str(d / "choice.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "shim.cpp"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    L, i = ctypes.c_long, ctypes.c_int
    for name, args, res in (("sizes", [i], i), ("choice", [i] + [L] * 5, i),
                            ("before", [i] + [L] * 4, L), ("tiles", [i, i] + [L] * 4, L),
                            ("threads", [i, i] + [L] * 4, L)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    return lib


def parts(rule, exact, R, E, N, K):
    """(rows, choice) of every launch of a call"""
    first = rule.before(exact, R, E, N, K)
    assert 0 < first <= R
    rows = [first] if first == R else [first, R - first]
    return [(r, rule.choice(exact, R if E else r, E, N, K, r)) for r in rows]


def check(rule, exact, R, E, N, K):
    got = parts(rule, exact, R, E, N, K)
    some = any(rule.threads(exact, i, R, E, N, R) < 2 ** 32 for i in range(rule.sizes(exact)))
    for r, c in got:
        if c < 0:  # the whole call is refused, and only where no tile takes it
            assert len(got) == 1 and not some, (R, E, N, K)
        else:
            assert rule.threads(exact, c, r if not E else R, E, N, r) < 2 ** 32, (R, E, N, K)


@pytest.mark.parametrize("exact", [0, 1])
def test_every_launch_fits_a_grid(rule, exact):
    """Outputs of 5 to some thousand rows by up to 2^30, as far as a card's memory holds them, and
    ordinary ones."""
    rng = np.random.default_rng(exact)
    size = 4 if exact else 2
    n = 0
    while n < 30000:
        N, R = int(2 ** rng.uniform(24, 30)), int(2 ** rng.uniform(2.4, 11))
        if N * R * size + 16 * N > 300e9:
            continue
        n += 1
        check(rule, exact, R, 0, N, 16)
    for _ in range(5000):
        check(rule, exact, int(2 ** rng.uniform(2.4, 20)), 0, int(2 ** rng.uniform(0, 20)),
              16 * int(2 ** rng.uniform(0, 13)))
        E = int(2 ** rng.uniform(0, 16))
        check(rule, exact, int(2 ** rng.uniform(3.5, 24)), E, int(2 ** rng.uniform(0, 24)), 1024)


@pytest.mark.parametrize("exact,R,N", [(1, 129, 537491005), (1, 132, 538781411), (0, 257, 551973648),
                                       (0, 5, 537866626), (1, 5, 538677395)])
def test_calls_whose_fastest_tiles_no_grid_takes(rule, exact, R, N):
    """The rest of the rows, or all of them, would by time alone take tiles of 8 waves or more, of
    which there would be too many."""
    check(rule, exact, R, 0, N, 16)
    assert all(c >= 0 for _, c in parts(rule, exact, R, 0, N, 16))


def test_calls_that_no_tile_takes_are_refused(rule):
    for exact in (0, 1):
        assert parts(rule, exact, 2 ** 30, 0, 2 ** 30, 16)[0][1] == -1
        check(rule, exact, 2 ** 30, 0, 2 ** 30, 16)


@pytest.mark.parametrize("exact", [0, 1])
def test_every_tile_is_taken(rule, exact):
    seen = {c for R in list(range(5, 70, 3)) + list(range(70, 4200, 67)) for N in range(64, 9000, 128)
            for _, c in parts(rule, exact, R, 0, N, 7168)}
    assert seen == set(range(rule.sizes(exact)))
