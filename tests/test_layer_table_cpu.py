"""Where a chunk of a packed batch lies (csrc/scan_table.hpp's locate), in a CPU build: right plans, wrong ones, and
the places the selective recurrence's gradients keep states at (csrc/selective.hip), which have to be the
sequence's own and inside what is set aside for them."""
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
extern "C" int table_locate(const int32_t* p, int seqs, int total, int cap, int c, int* out) {
  return ssm::ScanPlan{p, seqs, total, cap}.locate(c, out[0], out[1], out[2], out[3]);
}
extern "C" int table_capacity(int total, int seqs) { return ssm::scan_capacity(total, seqs); }
"""
CT, HB = 64, 8  # tokens of a chunk, and between two kept states


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("locate")
    (d / "table.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-static-libubsan", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sketched_recurrent_state_amd", "csrc"), str(d / "table.cpp"),
                    "-o", str(d / "table.so")], check=True)
    return ctypes.CDLL(str(d / "table.so"))


def plan(lib, lens):
    total, cap = sum(lens), lib.table_capacity(sum(lens), len(lens))
    start = np.concatenate([[0], np.cumsum(lens)])
    chunk = np.concatenate([[0], np.cumsum((np.asarray(lens) + CT - 1) // CT)])
    seq = np.full(cap, -1)
    for s in range(len(lens)):
        seq[chunk[s]:chunk[s + 1]] = s
    return np.concatenate([start, chunk, seq]).astype(np.int32), total, cap


def locate(lib, p, seqs, total, cap, c):
    out = (ctypes.c_int * 4)()
    return tuple(out) if lib.table_locate(p.ctypes.data_as(ctypes.c_void_p), seqs, total, cap, c, out) else None


def kept(first, length, pos):
    """Rows of a chunk's kept states: before every HB tokens of its sequence but the first."""
    end = min(pos + CT, length)
    return [first // HB + t // HB - 1 for t in range(pos, end, HB) if t > 0]


@pytest.mark.parametrize("lens", [[1], [64], [65], [7, 8, 9, 1, 0, 63, 64, 200], [0, 0, 5], [129, 0, 0, 15, 17],
                                  [1] * 20, [8] * 9, [9] * 9, [8003]])
def test_chunks_of_a_plan(lib, lens):
    p, total, cap = plan(lib, lens)
    want, c = [], 0
    for s, n in enumerate(lens):
        for pos in range(0, n, CT):
            want.append((s, sum(lens[:s]), n, pos))
    got = [locate(lib, p, len(lens), total, cap, c) for c in range(cap)]
    assert [g for g in got if g] == want and all(g is None for g in got[len(want):])
    rows = [r for _, first, n, pos in want for r in kept(first, n, pos)]
    assert len(set(rows)) == len(rows)  # no two states at one place
    assert all(0 <= r < total // HB + 1 for r in rows)


def test_wrong_plans_stay_inside(lib):
    rng = np.random.default_rng(11)
    seen = 0
    for _ in range(2000):
        lens = [int(n) for n in rng.integers(0, 200, rng.integers(1, 6))]
        p, total, cap = plan(lib, lens)
        for i in rng.choice(p.size, min(p.size, rng.integers(1, 4)), replace=False):
            p[i] = rng.choice([-2 ** 31, -65, -1, 0, 1, 63, 64, 200, 2 ** 31 - 1, int(p[i]) + 1, int(p[i]) - 1])
        for c in range(cap):
            g = locate(lib, p, len(lens), total, cap, c)
            if g is None:
                continue
            seen += 1
            s, first, n, pos = g
            assert 0 <= s < len(lens) and 0 <= first and 0 <= pos < n and first + n <= total and pos % CT == 0
            assert all(0 <= r < total // HB + 1 for r in kept(first, n, pos))
    assert seen > 2000
