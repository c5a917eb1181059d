"""CPU checks of the dense latent decode's plan (csrc/mla_dense_plan.h, compiled here for the host): the ranges
cover every block once, and no output is staged over a ring half that an earlier output's store may still read.

The ring has two halves; block x of a range (counted over its requests) is loaded into half x % 2.  A request's
output is staged in the half of its last block, or, as a partial, over both.  Its store is known to have read it
only when a later block has been loaded into that half."""
import ctypes
import subprocess

import numpy as np
import pytest

SOURCE = r"""
#include "mla_dense_plan.h"
using namespace dsa;
extern "C" {
int units(int blocks) { return units_of(blocks); }
int cut(int n, int total, int g) { return Ranges(n, total).cut(g); }
int settled(int c, int u, int blocks) { return settled_cut(c, u, blocks); }
int over_the_ring(int last, int blocks, int so_far) { return stage_whole_ring(last != 0, blocks, so_far) ? 1 : 0; }
int split_rule() { return kMlaSegUnits; }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from sparse_attention_paged_dsa_gb300 import build
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    return ctypes.CDLL(str(d / "plan.so"))


def ranges_of(plan, seqs, groups):
    """Per range: its requests as (request, first block, end block, blocks of the request, nothing follows)."""
    blocks = [-(-(-(-max(s, 0) // 4)) // 64) for s in seqs]
    starts = np.concatenate([[0], np.cumsum([plan.units(n) for n in blocks])]).tolist()
    total = starts[-1]
    n = max(min(groups, total), 1)

    def cut(g):
        c = plan.cut(n, total, g)
        if c >= total:
            return total
        b = int(np.searchsorted(starts, c, side="right")) - 1   # the request whose units hold it
        return plan.settled(c, starts[b], blocks[b])

    out = []
    for g in range(n):
        lo, hi, items = cut(g), cut(g + 1), []
        b = int(np.searchsorted(starts, lo, side="right")) - 1
        while b < len(seqs) and starts[b] < hi:
            base = starts[b] + plan.split_rule()
            blo, bhi = max(lo, base) - base, min(hi, starts[b + 1]) - base
            if blocks[b] > 0 and bhi > blo:
                items.append((b, blo, bhi, blocks[b], b + 1 >= len(seqs) or starts[b + 1] >= hi))
            b += 1
        out.append(items)
    return out, blocks


def unordered(ranges, over_the_ring):
    """Stagings over a half whose last staged output no load has replaced."""
    found = 0
    for items in ranges:
        pending, so_far = [False, False], 0
        for _, blo, bhi, nb, last in items:
            for x in range(so_far, so_far + bhi - blo):
                pending[x % 2] = False
            so_far += bhi - blo
            own = (so_far - 1) % 2
            whole = blo == 0 and bhi == nb
            halves = (0, 1) if not whole and over_the_ring(last, bhi - blo, so_far) else (own,)
            found += any(pending[h] for h in halves)
            for h in halves:
                pending[h] = True
    return found


# 152 ranges of one token; two, three and four tokens share 76, 50 and 38
@pytest.mark.parametrize("groups", [152, 76, 50, 38, 1])
@pytest.mark.parametrize("seqs", [[8192] * 64, [4096] * 200, [2048] * 300, [131072] * 64, [1 << 20], [1], [0, 0]])
def test_plan_of_equal_requests(plan, seqs, groups):
    check(plan, seqs, groups)


@pytest.mark.parametrize("groups", [152, 38])
@pytest.mark.parametrize("seed", range(12))
def test_plan_of_mixed_requests(plan, seed, groups):
    rng = np.random.default_rng(seed)
    batch = int(rng.integers(1, 400))
    check(plan, np.exp(rng.uniform(0, np.log(40000), batch)).astype(int).tolist(), groups)


def check(plan, seqs, groups):
    ranges, blocks = ranges_of(plan, seqs, groups)
    done = [0] * len(seqs)
    for items in ranges:
        for i, (b, blo, bhi, _, last) in enumerate(items):
            assert blo == done[b]
            done[b] = bhi
            assert not last or i == len(items) - 1
    assert done == blocks
    assert unordered(ranges, plan.over_the_ring) == 0


@pytest.mark.parametrize("seqs, groups", [([8192] * 64, 152), ([4096] * 200, 152), ([2048] * 300, 152),
                                          ([8192] * 64, 76), ([2048] * 301, 50), ([8192] * 64, 38)])
def test_plan_reaches_a_single_block_behind_another_request(plan, seqs, groups):
    """What the rule is for: staging over the ring whenever nothing follows would be unordered in these batches."""
    assert unordered(ranges_of(plan, seqs, groups)[0], lambda last, blocks, so_far: last) > 0
