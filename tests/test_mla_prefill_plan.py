"""CPU checks of how the prompt attention cuts rows into units (csrc/mla_prefill_plan.h, compiled here for the
host): every row of every head is in one unit, and no batch has more units than the launch allows for."""
import ctypes
import subprocess

import numpy as np
import pytest

SOURCE = r"""
#include "mla_prefill_plan.h"
using namespace dsa;
extern "C" {
int units(int rows, int live, int heads) { return Cut(rows, live, heads).units(); }
int rows_covered(int rows, int live, int heads) {
    const Cut c(rows, live, heads);
    const int behind = rows - c.long_blocks * kPrefillBlock;  // of the blocks of 256, which lie behind
    if (c.pair_blocks > 0 && (c.pair_blocks - 1) * kPrefillPair >= behind) return -1;  // one without rows
    return c.long_blocks * kPrefillBlock + c.pair_blocks * kPrefillPair;
}
long long most(long long q_rows, int batch, int heads) { return prefill_most_units(prefill_slots(q_rows, batch), heads); }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from sparse_attention_paged_dsa_gb300 import build
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    lib.most.argtypes, lib.most.restype = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int], ctypes.c_longlong
    return lib


@pytest.mark.parametrize("heads", [1, 2, 3, 4, 5, 7, 33, 127, 128])
@pytest.mark.parametrize("live", [0, 100, 768, 769, 50000])
def test_plan_of_one_request(plan, heads, live):
    for rows in range(2100):
        assert plan.rows_covered(rows, live, heads) >= rows
        assert plan.units(rows, live, heads) <= plan.most(rows, 1, heads)


def test_plan_of_an_odd_head(plan):
    """400 rows of 5 heads: two blocks of 256 rows, three units each."""
    assert plan.units(400, 400, 5) == 6 <= plan.most(400, 1, 5)
    assert plan.units(400, 400, 3) == 4 <= plan.most(400, 1, 3)


@pytest.mark.parametrize("seed", range(20))
def test_plan_of_batches(plan, seed):
    rng = np.random.default_rng(seed)
    batch, heads = int(rng.integers(1, 1025)), int(rng.integers(1, 129))
    rows = np.exp(rng.uniform(0, np.log(5000), batch)).astype(int) - 1
    live = np.exp(rng.uniform(0, np.log(5000), batch)).astype(int)
    units = sum(plan.units(int(r), int(n), heads) for r, n in zip(rows, live))
    assert units <= plan.most(int(rows.sum()), batch, heads)
