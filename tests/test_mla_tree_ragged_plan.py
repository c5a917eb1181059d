"""CPU checks of the tree decode's plan for trees of different sizes (csrc/mla_tree_plan.h, compiled here for the host):
each tile of four tokens is cut into ranges of its own; every range has one place in the order of work; every block of
every request and tile is done once, and its parts are where the merge looks for them."""
import ctypes
import subprocess

import numpy as np
import pytest

SOURCE = r"""
#include "mla_tree_plan.h"
using namespace dsa;
extern "C" {
int units_of(int seq, int drafted) { return tree_units(tree_blocks(tree_cache_pages(seq), drafted)); }
int cut(int n, int total, int g) { return Ranges(n, total).cut(g); }
int range_of(int n, int total, int unit) { return Ranges(n, total).of(unit); }
int settled(int c, int u, int blocks) { return tree_settled_cut(c, u, blocks); }
int tiles(int tokens) { return tree_tiles(tokens); }
int most(int tiles, int clusters) { return tree_ranges(tiles, clusters); }
int line_ranges(int total, int each) { return tree_line_ranges(total, each); }
int rank_of(const int* first, int tiles, int t, int g) { return tree_rank(first, tiles, t, g); }
long long cost(int units, int each, int tiles, int clusters) { return tree_cost_ragged(units, each, tiles, clusters); }
int seg() { return kTreeSegUnits; }
int whole() { return kTreeWholeBlocks; }
int rounds() { return kTreeMaxRounds; }
int max_ranges() { return kTreeMaxRanges; }
int max_units() { return kTreeMaxUnits; }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from sparse_attention_paged_dsa_gb300 import build
    d = tmp_path_factory.mktemp("tree_ragged_plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    lib.cost.restype = ctypes.c_longlong
    return lib


def lines(plan, seqs, counts, tokens):
    """Plan units of each request in each tile."""
    return [[plan.units_of(s, c) if 4 * t < c else 0 for s, c in zip(seqs, counts)] for t in range(plan.tiles(tokens))]


def choose(plan, line_units, clusters):
    """(ranges of each tile, the most that a call may have), as the kernel chooses them."""
    tiles = len(line_units)
    totals = [sum(u) for u in line_units]
    cap = plan.most(tiles, clusters) * tiles
    best = None
    for r in range(1, min(plan.max_ranges(), totals[0]) + 1):
        each = -(-totals[0] // r)
        n = [plan.line_ranges(t, each) for t in totals]
        if sum(n) <= cap:
            cost = (plan.cost(sum(n), each, tiles, clusters), r)
            best = min(best or (cost, n), (cost, n))
    return (best[1] if best else [0] * tiles), cap


def check(plan, seqs, counts, tokens, clusters):
    units = lines(plan, seqs, counts, tokens)
    n, cap = choose(plan, units, clusters)
    tiles = len(units)
    assert sum(n) <= cap <= min(plan.max_units(), plan.rounds() * max(clusters, tiles))
    first = (ctypes.c_int * (tiles + 1))(*np.concatenate([[0], np.cumsum(n)]).tolist())
    ranks = [plan.rank_of(first, tiles, t, g) for t in range(tiles) for g in range(n[t])]
    assert sorted(ranks) == list(range(sum(n)))
    for t in range(tiles):                                           # a tile's ranges come in order
        assert ranks[first[t]:first[t + 1]] == sorted(ranks[first[t]:first[t + 1]])
        assert n[t] <= plan.max_ranges() and (n[t] > 0) == (sum(units[t]) > 0)
        if n[t] == 0:
            continue
        starts, total = np.concatenate([[0], np.cumsum(units[t])]).tolist(), sum(units[t])
        blocks = [u - plan.seg() if u else 0 for u in units[t]]

        def cut(g):
            c = plan.cut(n[t], total, g)
            if c >= total:
                return total
            b = int(np.searchsorted(starts, c, side="right")) - 1
            return plan.settled(c, starts[b], blocks[b])

        done, parts = [0] * len(seqs), [[] for _ in seqs]
        for g in range(n[t]):
            lo, hi = cut(g), cut(g + 1)
            b = max(int(np.searchsorted(starts, lo, side="right")) - 1, 0)
            while b < len(seqs) and starts[b] < hi:
                base = starts[b] + plan.seg()
                blo, bhi = max(lo, base) - base, min(hi, starts[b + 1]) - base
                if bhi > blo:
                    assert blo == done[b]
                    done[b] = bhi
                    parts[b].append(g)
                b += 1
        assert done == blocks
        for b, k in enumerate(blocks):
            if k <= plan.whole():
                assert len(parts[b]) <= 1
            else:
                assert parts[b] == list(range(plan.range_of(n[t], total, starts[b] + plan.seg()),
                                              plan.range_of(n[t], total, starts[b + 1] - 1) + 1))


@pytest.mark.parametrize("seed", range(40))
def test_ragged_plan(plan, seed):
    rng = np.random.default_rng(seed)
    batch, tokens = int(rng.integers(1, 300)), int(rng.integers(2, 65))
    seqs = np.exp(rng.uniform(0, np.log(300000), batch)).astype(int).tolist()
    counts = rng.integers(0, tokens + 1, batch).tolist()
    check(plan, seqs, counts, tokens, int(rng.integers(16, 77)))


@pytest.mark.parametrize("counts", [[0] * 5, [64, 0, 0, 0, 0], [0, 0, 0, 0, 64], [4, 5, 8, 9, 64], [1] * 5, [64] * 5])
@pytest.mark.parametrize("clusters", [7, 36, 76])
def test_ragged_plan_few(plan, counts, clusters):
    check(plan, [0, 131072, 1, 5000, 100000], counts, 64, clusters)


def test_equal_trees_go_range_by_range(plan):
    for tiles in (1, 2, 7, 16):
        for n in (1, 5, 31):
            first = (ctypes.c_int * (tiles + 1))(*[t * n for t in range(tiles + 1)])
            assert [plan.rank_of(first, tiles, t, g) for g in range(n) for t in range(tiles)] == list(range(n * tiles))


def test_small_trees_cost_little(plan):
    """Half of the tokens take little more than half of the time of all, by the plan's count."""
    rng = np.random.default_rng(1)
    for batch, tokens, seq in [(64, 32, 16384), (32, 16, 32768), (8, 64, 32768)]:
        counts = rng.integers(0, tokens + 1, batch).tolist()
        units = lines(plan, [seq] * batch, counts, tokens)
        n, _ = choose(plan, units, 36)
        longest = max(-(-sum(u) // k) for u, k in zip(units, n) if k) * -(-sum(n) // 36)
        assert longest * 36 <= 1.25 * sum(map(sum, units))
