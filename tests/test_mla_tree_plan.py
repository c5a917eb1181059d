"""CPU checks of the tree decode's plan (csrc/mla_tree_plan.h, compiled here for the host): the units cover every
block of every request and tile once, partial outputs are where the merge looks for them, and the number of
ranges is within what the workspace holds."""
import ctypes
import subprocess

import numpy as np
import pytest

SOURCE = r"""
#include "mla_tree_plan.h"
using namespace dsa;
extern "C" {
int cache_pages(int tokens) { return tree_cache_pages(tokens); }
int blocks(int pages, int drafted) { return tree_blocks(pages, drafted); }
int units(int blocks) { return tree_units(blocks); }
int cut(int n, int total, int g) { return Ranges(n, total).cut(g); }
int range_of(int n, int total, int unit) { return Ranges(n, total).of(unit); }
int settled(int c, int u, int blocks) { return tree_settled_cut(c, u, blocks); }
int tiles(int tokens) { return tree_tiles(tokens); }
int most(int tiles, int clusters) { return tree_ranges(tiles, clusters); }
long long cost(int r, int total, int tiles, int clusters, int tokens) { return tree_cost(r, total, tiles, clusters, tokens); }
int seg() { return kTreeSegUnits; }
int whole() { return kTreeWholeBlocks; }
int rounds() { return kTreeMaxRounds; }
int max_ranges() { return kTreeMaxRanges; }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from sparse_attention_paged_dsa_gb300 import build
    d = tmp_path_factory.mktemp("tree_plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    lib.cost.restype = ctypes.c_longlong
    return lib


def check(plan, seqs, counts, tokens, clusters):
    tiles = plan.tiles(tokens)
    most = plan.most(tiles, clusters)
    assert 1 <= most <= plan.max_ranges() and most * tiles <= plan.rounds() * max(clusters, tiles)
    blocks = [plan.blocks(plan.cache_pages(s), c) for s, c in zip(seqs, counts)]
    for s, c, n in zip(seqs, counts, blocks):
        pages = -(-(-(-s // 4)) // 64)
        assert n == (0 if c == 0 else -(-(pages + 1) // 2))       # two pages a block, the drafted one behind the others
    starts = np.concatenate([[0], np.cumsum([plan.units(n) for n in blocks])]).tolist()
    total = starts[-1]
    if total == 0:
        return
    n = min(range(1, min(most, total) + 1), key=lambda r: (plan.cost(r, total, tiles, clusters, tokens), r))

    def cut(g):
        c = plan.cut(n, total, g)
        if c >= total:
            return total
        b = int(np.searchsorted(starts, c, side="right")) - 1
        return plan.settled(c, starts[b], blocks[b])

    done, ranges_of = [0] * len(seqs), [[] for _ in seqs]
    for g in range(n):
        lo, hi = cut(g), cut(g + 1)
        b = max(int(np.searchsorted(starts, lo, side="right")) - 1, 0)
        while b < len(seqs) and starts[b] < hi:
            base = starts[b] + plan.seg()
            blo, bhi = max(lo, base) - base, min(hi, starts[b + 1]) - base
            if blocks[b] and bhi > blo:
                assert blo == done[b]
                done[b] = bhi
                ranges_of[b].append(g)
            b += 1
    assert done == blocks
    for b, n_b in enumerate(blocks):
        if n_b <= plan.whole():
            assert len(ranges_of[b]) <= 1                            # written whole, and not merged
        else:
            first = plan.range_of(n, total, starts[b] + plan.seg())
            last = plan.range_of(n, total, starts[b + 1] - 1)
            assert ranges_of[b] == list(range(first, last + 1))      # where the merge looks for its parts


@pytest.mark.parametrize("tokens", [3, 4, 5, 8, 16, 27, 32, 33, 64])
@pytest.mark.parametrize("clusters", [36, 38, 33, 7])
@pytest.mark.parametrize("seqs", [[131072] * 16, [8192] * 13, [1 << 20], [0], [0, 0, 5], [512] * 64, [1024] * 1024])
def test_plan_of_equal_requests(plan, seqs, tokens, clusters):
    check(plan, seqs, [tokens] * len(seqs), tokens, clusters)


@pytest.mark.parametrize("seed", range(24))
def test_plan_of_mixed_requests(plan, seed):
    rng = np.random.default_rng(seed)
    batch, tokens = int(rng.integers(1, 400)), int(rng.integers(3, 65))
    seqs = np.exp(rng.uniform(0, np.log(300000), batch)).astype(int).tolist()
    counts = rng.integers(0, tokens + 1, batch).tolist()
    check(plan, seqs, counts, tokens, int(rng.integers(16, 40)))


def test_ranges_fill_the_device_for_long_requests(plan):
    """With long requests the chosen ranges leave at most an eighth of the clusters' time unused."""
    for tokens in (3, 4, 8, 12, 16, 24, 27, 32, 48, 64):
        tiles, clusters, total = plan.tiles(tokens), 36, 64 * 520
        most = plan.most(tiles, clusters)
        n = min(range(1, most + 1), key=lambda r: (plan.cost(r, total, tiles, clusters, tokens), r))
        rounds = -(-n * tiles // clusters)
        assert total * tiles / (rounds * clusters * -(-total // n)) >= 7 / 8
