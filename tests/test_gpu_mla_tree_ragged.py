"""GPU tests of dsa_mla_tree_decode for trees of different sizes: each tile of four tokens is cut into ranges of its
own.  Cases, fp64 reference and tolerances as in test_gpu_mla_tree.py."""
from types import SimpleNamespace

import numpy as np
import pytest

from test_gpu_mla_tree import Case, run, tree
from test_gpu_mla_tree_long import check_large_scores

pytestmark = pytest.mark.gpu

WIDE = 1 << 18


def ragged(seqs, counts, tokens, seed, context=WIDE, **kw):
    rng = np.random.default_rng(seed)
    case = Case(seqs, context, tokens, counts=counts, seed=seed, masks=[tree(rng, tokens, back=5) for _ in seqs], **kw)
    for b, c in enumerate(counts):
        case.draft[b, max(c, 0):] = float("nan")
        case.q[b, max(c, 0):] = float("nan")
    return case


@pytest.mark.parametrize("counts", [[64, 0, 0, 0, 0], [0, 0, 0, 0, 64], [4, 5, 8, 9, 64], [1] * 5, [64, 1, 1, 1, 1],
                                    [33, 0, 60, 0, 3]])
def test_ragged_few(gpu_lib, counts):
    case = ragged([0, 70000, 1, 5000, 30000], counts, 64, seed=sum(counts))
    case.check(*run(gpu_lib, case), untouched=7.0)


@pytest.mark.parametrize("batch, tokens, longest", [(40, 32, 16384), (64, 12, 8192), (100, 9, 3000), (300, 5, 2000),
                                                    (1024, 6, 900), (12, 64, 30000), (2, 13, 100000)])
def test_ragged_batches(gpu_lib, batch, tokens, longest):
    """More and fewer rows than places for partial outputs."""
    rng = np.random.default_rng(batch)
    seqs = np.exp(rng.uniform(0, np.log(longest), batch)).astype(int)
    seqs[: batch // 3] = longest - np.arange(batch // 3)
    counts = rng.integers(0, tokens + 1, batch).tolist()
    case = ragged(seqs.tolist(), counts, tokens, seed=batch, context=WIDE if batch <= 100 else 1 << 13)
    case.check(*run(gpu_lib, case), untouched=7.0, rows=None if batch <= 12 else rng.choice(batch, 12, replace=False).tolist())


def test_ragged_done_again(gpu_lib):
    """Scores far above the first block's in one tile: the whole call is done again."""
    case = Case([6000, 30000, 900, 0, 12000], WIDE, 18, counts=[18, 3, 7, 18, 12], seed=3, scale=1.0 / 24.0)
    case.draft[4, 9] *= 512.0
    out, lse = run(gpu_lib, case)
    for b, count in enumerate(case.counts):
        check_large_scores(SimpleNamespace(tokens=count, scale=case.scale, q=case.q, entries=case.entries), out, lse, [b])


def test_ragged_replayed(gpu_lib):
    """A replayed call takes new counts and lengths, and has the bits of a call of its own."""
    import torch
    case = ragged([30000, 900, 0, 65536, 20000], [9, 2, 5, 1, 7], 9, seed=12)
    case.q.nan_to_num_(nan=1.0)
    case.draft.nan_to_num_(nan=1.0)
    ws = gpu_lib.new_tree_workspace(5, 9)
    counts = torch.tensor([9, 2, 5, 1, 7], dtype=torch.int32).cuda()
    out, lse = torch.empty_like(case.q[..., :512]).contiguous(), torch.empty(5, 9, 64, device="cuda")
    call = lambda ws, **kw: gpu_lib.dsa_mla_tree_decode(*case.args(), token_counts=counts, workspace=ws, **kw)  # noqa: E731
    call(ws, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(ws, out=out, lse=lse)
    for new in ([9, 2, 5, 1, 7], [0, 9, 9, 0, 1], [4, 4, 4, 4, 4], [0, 0, 0, 0, 0], [9, 9, 9, 9, 9]):
        counts.copy_(torch.tensor(new, dtype=torch.int32))
        out.zero_()
        lse.zero_()
        graph.replay()
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        call(gpu_lib.new_tree_workspace(5, 9), out=o, lse=l)
        assert torch.equal(out, o) and torch.equal(lse, l)
    assert gpu_lib.get_error(ws) == 0


@pytest.mark.parametrize("seed", range(12))
def test_ragged_random(gpu_lib, seed):
    rng = np.random.default_rng(3000 + seed)
    batch, tokens = int(rng.integers(2, 60)), int(rng.integers(2, 65))
    seqs = np.exp(rng.uniform(0, np.log(9000 if batch > 8 else 60000), batch)).astype(int).tolist()
    case = ragged(seqs, rng.integers(0, tokens + 1, batch).tolist(), tokens, seed=seed, context=1 << int(rng.integers(16, 20)))
    case.check(*run(gpu_lib, case), untouched=7.0, rows=rng.choice(batch, min(batch, 12), replace=False).tolist())
