"""The checks that keep the scan inside its arrays whatever a plan holds (csrc/scan_table.hpp), in a
CPU build: plausible but wrong entries, one for each bound, and random tables."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include "scan_table.hpp"
extern "C" int table_cell(const int32_t* p, int seqs, int total, int cap, int c, int* out) {
  return ssm::ScanPlan{p, seqs, total, cap}.cell(c, out[0], out[1]);
}
extern "C" int table_sequence(const int32_t* p, int seqs, int total, int cap, int s, int* out) {
  return ssm::ScanPlan{p, seqs, total, cap}.sequence(s, out[0], out[1], out[2]);
}
extern "C" int table_capacity(int total, int seqs) { return ssm::scan_capacity(total, seqs); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("table")
    (d / "table.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-static-libubsan", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sketched_recurrent_state_amd", "csrc"), str(d / "table.cpp"),
                    "-o", str(d / "table.so")], check=True)
    return ctypes.CDLL(str(d / "table.so"))


class Table:
    def __init__(self, lib, lens, total=None):
        self.lib, self.n = lib, len(lens)
        self.total = sum(lens) if total is None else total
        self.cap = lib.table_capacity(self.total, self.n)
        start = np.concatenate([[0], np.cumsum(lens)])
        chunk = np.concatenate([[0], np.cumsum((np.asarray(lens) + 63) // 64)])
        seq = np.full(self.cap, -1)
        for s in range(self.n):
            seq[chunk[s]:chunk[s + 1]] = s
        self.p = np.concatenate([start, chunk, seq]).astype(np.int32)
        # views: a change is a change of the plan
        self.start, self.chunk, self.seq = np.split(self.p, [self.n + 1, 2 * self.n + 2])

    def _call(self, f, i, k):
        out = (ctypes.c_int * k)()
        ok = f(self.p.ctypes.data_as(ctypes.c_void_p), self.n, self.total, self.cap, i, out)
        return tuple(out) if ok else None

    def cell(self, c):
        return self._call(self.lib.table_cell, c, 2)

    def sequence(self, s):
        return self._call(self.lib.table_sequence, s, 3)


def in_bounds(t):
    """Whether everything the kernels would touch is inside: tokens, and the workspace's cells."""
    for c in range(t.cap):
        got = t.cell(c)
        if got and not (0 <= got[0] and 1 <= got[1] <= 64 and got[0] + got[1] <= t.total):
            return False
    for s in range(t.n):
        got = t.sequence(s)
        if got:
            tok, length, first = got
            if not (0 <= tok and 0 <= length and tok + length <= t.total and 0 <= first
                    and first + (length + 63) // 64 <= t.cap):
                return False
    return True


def test_a_plan_names_every_token_once(lib):
    for lens in ([], [0], [1], [64], [65, 0, 0, 130, 63], [200]):
        t = Table(lib, lens, sum(lens) + 7)
        seen = np.zeros(t.total, int)
        for c in range(t.cap):
            got = t.cell(c)
            if got:
                seen[got[0]:got[0] + got[1]] += 1
        assert (seen[:sum(lens)] == 1).all() and (seen[sum(lens):] == 0).all()
        first = 0
        for s, n in enumerate(lens):
            assert t.sequence(s) == (sum(lens[:s]), n, first)
            first += (n + 63) // 64


BIG = 2 ** 31 - 1
# what is changed in the plan of lengths 100, 70, 30 (starts 0 100 170 200, chunks 0 2 4 5, table
# 0 0 1 1 2 -1), then the chunks and the sequences that must be refused for it
WRONG = {
    "a sequence that ends past the arrays": (lambda t: t.start.__setitem__(3, 201), [4], [2]),
    "far past the arrays": (lambda t: t.start.__setitem__(3, BIG), [4], [2]),
    "starts in descending order": (lambda t: t.start.__setitem__(1, 180), [2, 3], [1]),
    "a start below zero": (lambda t: t.start.__setitem__(0, -1), [0, 1], [0]),
    "a start far below zero": (lambda t: t.start.__setitem__(0, -BIG - 1), [0, 1], [0]),
    "an end below zero": (lambda t: t.start.__setitem__(1, -5), [0, 1, 2, 3], [0, 1]),
    "chunks past the table": (lambda t: t.chunk.__setitem__(1, 5), [2, 3], [1]),
    "chunks far past the table": (lambda t: t.chunk.__setitem__(1, BIG), [2, 3], [1]),
    "chunks below zero": (lambda t: t.chunk.__setitem__(2, -1), [4], [2]),
    "chunks far below zero": (lambda t: t.chunk.__setitem__(2, -BIG - 1), [4], [2]),
    "a chunk of a sequence that starts later": (lambda t: t.seq.__setitem__(3, 2), [3], []),
    "a chunk of one that starts much later": (lambda t: t.seq.__setitem__(0, 2), [0], []),
    "a chunk of a sequence that has ended": (lambda t: t.seq.__setitem__(4, 0), [4], []),
    "a chunk of no sequence": (lambda t: t.seq.__setitem__(1, 3), [1], []),
    "a chunk of a sequence far off": (lambda t: t.seq.__setitem__(1, BIG), [1], []),
    "a chunk of a sequence below zero": (lambda t: t.seq.__setitem__(1, -2), [1], []),
}


@pytest.mark.parametrize("name", WRONG)
def test_wrong_entries_are_refused(lib, name):
    change, chunks, sequences = WRONG[name]
    t = Table(lib, [100, 70, 30])
    before = [t.cell(c) for c in range(t.cap)], [t.sequence(s) for s in range(t.n)]
    assert t.cap == 6 and None not in before[0][:5] + before[1]
    change(t)
    for c in chunks:
        assert t.cell(c) is None
    for s in sequences:
        assert t.sequence(s) is None
    assert in_bounds(t)


def test_random_tables_stay_in_bounds(lib):
    rng = np.random.default_rng(0)
    accepted = 0
    for _ in range(4000):
        lens = rng.integers(0, 200, rng.integers(1, 6)).tolist()
        t = Table(lib, lens, sum(lens) + int(rng.integers(0, 70)))
        for _ in range(rng.integers(1, 8)):
            i = rng.integers(len(t.p))
            x = rng.choice([int(t.p[i]) + rng.integers(-3, 4), rng.integers(-70, t.total + 70),
                            rng.choice([BIG, -BIG - 1, -1, t.total, t.cap, t.n]),
                            t.p[rng.integers(len(t.p))]])
            t.p[i] = min(max(int(x), -BIG - 1), BIG)
        assert in_bounds(t)
        accepted += sum(t.cell(c) is not None for c in range(t.cap))
    assert accepted > 4000
