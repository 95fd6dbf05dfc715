"""Which state a sequence of a selective prompt begins with (csrc/scan_table.hpp's goes_on), in a CPU build: where
states are continued in place, the pass that writes them reads none that another group of chunks writes."""
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
