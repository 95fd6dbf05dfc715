"""Which state a sequence of a selective prompt begins with (csrc/scan_table.hpp's goes_on), in a CPU build: where
states are continued in place, the pass that writes them reads none that another group of chunks writes. And where its
gradients keep states (kept_place, kept_places, which the kernels and the workspace's size are made of)."""
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
extern "C" int table_goes_on(int c, int len, int e1, int cap) { return ssm::goes_on(c, len, e1, cap); }
extern "C" int table_kept(int first, int pos) { return ssm::kept_place(first, pos); }
extern "C" int table_kept_places(int total) { return ssm::kept_places(total); }
extern "C" int table_kept_tokens() { return ssm::KT; }
extern "C" int table_locate(const int32_t* p, int seqs, int total, int cap, int c, int* out) {
  return ssm::ScanPlan{p, seqs, total, cap}.locate(c, out[0], out[1], out[2], out[3]);
}
"""
CT = 64


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("groups")
    (d / "table.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-static-libubsan", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sketched_recurrent_state_amd", "csrc"), str(d / "table.cpp"),
                    "-o", str(d / "table.so")], check=True)
    return ctypes.CDLL(str(d / "table.so"))


def accesses(lib, lens, size):
    """Groups of `size` entries: of every sequence (group that begins it, group that ends it, whether the first reads
    the local pass's copy, whether that pass makes one there)."""
    cap = sum(lens) // CT + len(lens)
    first = np.concatenate([[0], np.cumsum([-(-n // CT) for n in lens])])
    for s, n in enumerate(lens):
        if n == 0:
            continue
        begins, ends = int(first[s]) // size, (int(first[s + 1]) - 1) // size
        e1 = min((begins + 1) * size, cap)
        copied = bool(lib.table_goes_on(int(first[s]), n, e1, cap))
        # the local pass keeps the start of the sequence that holds the group's last used entry and goes on
        last = max(t for t in range(len(lens)) if lens[t] > 0 and first[t] < e1)
        yield begins, ends, copied, last == s and first[s + 1] > e1


@pytest.mark.parametrize("size", [1, 2, 3, 9, 1000])
def test_no_state_is_read_in_one_group_and_written_in_another(lib, size):
    rng = np.random.default_rng(size)
    batches = [[64] + [128] * 40, [200] * 64, [100] * 64, [1], [64], [65], [0, 0, 5], [63] * 9, [8003]]
    batches += [[int(n) for n in rng.integers(0, 400, rng.integers(1, 60))] for _ in range(200)]
    crossing = 0
    for lens in batches:
        for begins, ends, copied, made in accesses(lib, lens, size):
            assert copied == (begins != ends) == made
            crossing += copied
    assert crossing > 100 or size == 1000


def test_the_last_group_is_the_end(lib):
    """Nothing goes on behind the table, whatever a plan says: with one group there are no copies."""
    assert not lib.table_goes_on(0, 2 ** 31 - 1, 4, 4)
    assert lib.table_goes_on(0, 2 ** 31 - 1, 4, 5)
    assert not lib.table_goes_on(3, 64, 4, 5) and lib.table_goes_on(3, 65, 4, 5)
    assert lib.table_goes_on(2 ** 26, 2 ** 31 - 1, 2 ** 26 + 1, 2 ** 27)


def places(lib, first, length, begin=0, end=None):
    """Of a sequence's tokens [begin, end)."""
    step = lib.table_kept_tokens()
    assert CT % step == 0 and begin % CT == 0
    return [lib.table_kept(first, t) for t in range(begin, length if end is None else min(end, length), step) if t > 0]


@pytest.mark.parametrize("lens", [[1], [64], [65], [7, 8, 9, 1, 0, 63, 64, 200], [0, 0, 5], [129, 0, 0, 15, 17], [1] * 20,
                                  [8] * 9, [9] * 9, [15] * 7, [8003], None])
def test_kept_states_have_places_of_their_own(lib, lens):
    rng = np.random.default_rng(2)
    for lens in [lens] if lens else [[int(n) for n in rng.integers(0, 40, rng.integers(1, 50))] for _ in range(300)]:
        first = np.concatenate([[0], np.cumsum(lens)])
        got = [p for s, n in enumerate(lens) for p in places(lib, int(first[s]), n)]
        assert len(set(got)) == len(got)
        assert all(0 <= p < lib.table_kept_places(sum(lens)) for p in got)


def test_kept_states_of_wrong_plans_stay_inside(lib):
    rng = np.random.default_rng(12)
    out, seen = (ctypes.c_int * 4)(), 0
    for _ in range(1500):
        lens = rng.integers(0, 200, rng.integers(1, 6))
        total, n = int(lens.sum()), len(lens)
        cap = total // CT + n
        chunk = np.concatenate([[0], np.cumsum((lens + CT - 1) // CT)])
        seq = np.concatenate([np.repeat(np.arange(n), np.diff(chunk)), np.full(cap - chunk[-1], -1)])
        p = np.concatenate([[0], np.cumsum(lens), chunk, seq]).astype(np.int32)
        for i in rng.choice(p.size, min(p.size, 3), replace=False):
            p[i] = rng.choice([-2 ** 31, -1, 0, 1, 63, 64, 200, 2 ** 31 - 1, int(p[i]) + 1, int(p[i]) - 1])
        for c in range(cap):
            if lib.table_locate(p.ctypes.data_as(ctypes.c_void_p), n, total, cap, c, out):
                _, first, length, pos = out
                seen += 1
                assert all(0 <= k < lib.table_kept_places(total) for k in places(lib, first, length, pos, pos + CT))
    assert seen > 1500
