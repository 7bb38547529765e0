"""What the reordering decides on the host, compiled by itself: no GPU. Whether states share memory, against their bytes
counted one by one; which states are the same; how many units of work there are."""
import ctypes
import itertools
import os
import random
import shutil
import subprocess

import pytest

from gradient_row_online_gb300 import build as B
from gradient_row_online_gb300 import headloss as hlb

DRIVER = """
#include "hl_reorder_plan.h"
extern "C" int overlap(const headloss_state* s, int n, int64_t rows) { return hl_reorder::conflict(s, n, rows); }
extern "C" int distinct(const headloss_state* s, int n, headloss_state* to) { return hl_reorder::without_repeats(s, n, to); }
extern "C" int64_t shares(int64_t lines, int64_t most, int64_t chunks, int64_t grid) { return hl_reorder::shares_of(lines, most, chunks, grid); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    folder = tmp_path_factory.mktemp("plan")
    source, lib = folder / "driver.cpp", folder / "driver.so"
    source.write_text(DRIVER)
    compiler = shutil.which("g++") or shutil.which("c++")
    subprocess.run([compiler, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-Wno-pedantic", "-shared", "-fPIC", "-I" + B.CSRC, "-I" + B.INCLUDE,
                    str(source), "-o", str(lib)], check=True)
    lib = ctypes.CDLL(str(lib))
    lib.overlap.argtypes = [ctypes.POINTER(hlb.headloss_state), ctypes.c_int, ctypes.c_int64]
    lib.distinct.argtypes = [ctypes.POINTER(hlb.headloss_state), ctypes.c_int, ctypes.POINTER(hlb.headloss_state)]
    lib.shares.argtypes, lib.shares.restype = [ctypes.c_int64] * 4, ctypes.c_int64
    return lib


def table(*states):
    return (hlb.headloss_state * len(states))(*(hlb.headloss_state(*s) for s in states))


def taken(base, s, rows):
    _, _, outer, positions, run, rs, os_, ps = s
    return {base + i * rs + o * os_ + p * ps + k for i, o, p, k in
            itertools.product(range(rows), range(outer), range(positions), range(run))}


def expected(states, rows):
    """Whether a byte that one state writes is another's, or the same's in another place."""
    for i, s in enumerate(states):
        written = taken(s[1], s, rows)
        if s[0] != s[1] and written & taken(s[0], s, rows):
            return True
        for t in states[:i] + states[i + 1:]:
            if written & taken(t[0], t, rows) or written & taken(t[1], t, rows):
                return True
    return False


def test_random_layouts(plan):
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(4000):
        rows, n = rng.randint(1, 4), rng.randint(1, 3)
        nested = rng.random() < 0.6
        states = []
        outer, positions, run = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 5)
        steps = rng.sample([run * rng.randint(1, 3), run * positions * rng.randint(1, 3), run * positions * outer * rng.randint(1, 3)], 3)
        for _ in range(n):
            if not nested or rng.random() < 0.2:
                outer, positions, run = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 5)
                steps = [rng.randint(0, 40) for _ in range(3)]
            state = 1000 + rng.randint(0, 150)
            out = state if rng.random() < 0.5 else 1000 + rng.randint(0, 150)
            states.append((state, out, outer, positions, run, *steps))
        want = expected(states, rows)
        assert bool(plan.overlap(table(*states), n, rows)) == want, (rows, states)
        seen[want] += 1
    assert min(seen) > 400


def test_caches_as_programs_hold_them(plan):
    """Keys and values in one buffer, of one layer and of all, in every order of the dimensions; the same with a row too many."""
    heads, positions, width, layers, rows = 4, 512, 64, 24, 16
    one = positions * width

    def state(at, rs, os_, ps, w=width, p=positions):
        return (1 << 20 | 0) + at, (1 << 20) + at, heads, p, w, rs, os_, ps
    layouts = {
        "rows first": [state(j * heads * one, layers * heads * one, one, width) for j in range(layers)],
        "layers first": [state(j * rows * heads * one, heads * one, one, width) for j in range(layers)],
        "keys beside values": [state(j * width, heads * positions * 2 * width, positions * 2 * width, 2 * width) for j in range(2)],
        "positions first": [state(j * width, layers * heads * width, layers * width, rows * layers * heads * width) for j in range(layers)],
        "keys wider": [state(0, heads * positions * 192, positions * 192, 192, 128), state(128, heads * positions * 192, positions * 192, 192, 64)],
        "halves of the positions": [state(0, heads * one, one, width, p=positions // 2),
                                    state(positions // 2 * width, heads * one, one, width, p=positions // 2)],
    }
    for name, states in layouts.items():
        assert not plan.overlap(table(*states), len(states), rows), name
        moved = list(states)
        moved[-1] = (states[-1][0] - 1, states[-1][1] - 1) + states[-1][2:]
        assert plan.overlap(table(*moved), len(moved), rows), name
    assert plan.overlap(table(*layouts["layers first"]), layers, rows + 1)


def test_outs_that_others_read(plan):
    a, b, c = 1 << 12, 2 << 12, 3 << 12
    layout = (1, 1, 64, 64, 0, 0)
    for states, want in (([(a, b), (b, a)], 1), ([(a, b), (b, c)], 1), ([(a, b), (a, c)], 0), ([(a, c), (b, c)], 1), ([(a, a), (a, b)], 1),
                         ([(a, b)], 0), ([(a, a)], 0), ([(a, a + 64)], 1), ([(a, a + 512)], 0)):
        assert plan.overlap(table(*(s + layout for s in states)), len(states), 8) == want, states


def test_many_states_and_layouts_that_do_not_nest(plan):
    states = [((i + 1) << 12, (i + 1) << 12, 1, 1, 4096 // 8, 4096 // 8, 0, 0) for i in range(200000)]
    assert not plan.overlap(table(*states), len(states), 8)
    assert plan.overlap(table(*states), len(states), 9)
    # even and odd bytes apart, whatever the strides; and a search that is too long is answered by yes
    apart = [(1 << 20, 1 << 20, 100, 100, 1, 2 * 10007, 2 * 101, 2), (1 + (1 << 20), 1 + (1 << 20), 100, 100, 1, 2 * 9973, 2 * 103, 2)]
    assert plan.overlap(table(*apart), 2, 100) in (0, 1)


def test_states_that_are_the_same(plan):
    s = [(4096, 4096, 2, 5, 8, 80, 40, 8), (4096, 4096, 2, 5, 16, 80, 40, 8), (8192, 4096, 2, 5, 8, 80, 40, 8), (4096, 4096, 1, 5, 8, 80, 7, 8),
         (4096, 4096, 1, 5, 8, 80, 9, 8)]
    order = [3, 0, 0, 1, 2, 0, 4, 1]
    to = (hlb.headloss_state * len(order))()
    n = plan.distinct(table(*(s[i] for i in order)), len(order), to)
    got = [tuple(getattr(e, f) for f, _ in hlb.headloss_state._fields_) for e in to[:n]]
    assert got == [s[3], s[0], s[1], s[2]]  # (a stride that nothing is stepped by makes no difference)
    assert plan.distinct(table(s[0]), 0, to) == 0


@pytest.mark.parametrize("grid", [1, 148, 152, 304, 608, 1216])
def test_units_are_counted_in_32_bits(plan, grid):
    for lines in (1, 7, 600, grid, 4 * grid, 1 << 20, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 31) - 600, (1 << 31) - 1):
        for most in (1, 4096, 8191, 8192, 1 << 20, 1 << 40):
            for chunk in (128, 768, 4096):
                shares = plan.shares(lines, most, -(-most // chunk), grid)
                assert 1 <= shares <= -(-most // chunk)
                assert lines * shares + grid < 1 << 32, (lines, most, chunk)  # where a CTA's last step leads
