"""GPU tests of dsa_mla_tree_decode: one request's values never change another's results.

Trees of more than two tokens in calls large enough for the kernel on clusters of four CTAs, which keeps no running
maximum: requests whose scores rise far above their first ones, or are NaN, are done a second time by another
kernel.  The order of a request's sums depends on the batch's lengths and counts only, so the other requests' bits
stay, and so do its own, whichever others are done again.  Values are compared as in test_gpu_mla_tree.py."""
import numpy as np
import pytest

from test_gpu_mla_tree import Case, run

pytestmark = pytest.mark.gpu

WIDE = 1 << 18


def far(case, b):
    """Makes request b's drafted entries, its last block, score far above the cache's (their keys grow 64-fold)."""
    case.draft[b] *= 64.0


def nan(case, b):
    case.q[b, 0, 3, 0] = float("nan")


def same(case, got, want, rows):
    import torch
    for b in rows:
        n = case.drafted(b)
        for g, w in zip(got, want):
            assert torch.equal(g[b, :n].view(torch.int16 if g.element_size() == 2 else torch.int32),
                               w[b, :n].view(torch.int16 if w.element_size() == 2 else torch.int32)), b


def check_far(case, out, lse, b):
    """Request b against fp64, with the slack that scores of thousands have (as in test_tree_running_max)."""
    import torch
    for j in range(case.drafted(b)):
        kv = case.entries(b, j)
        s = case.scale * (case.q[b, j].double() @ kv.T)
        size = case.scale * (case.q[b, j].double().abs() @ kv.abs().T)
        slack = float((size * 2.0 ** -21).max())
        w = torch.softmax(s, dim=1)
        o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
        tol = (2.0 ** -8 + 2.0 ** -10 + 2 * slack) * a + 2.0 ** -8 * o.abs() + 1e-12
        assert not ((out[b, j].double() - o).abs() > tol).any(), (b, j)
        l = torch.logsumexp(s, 1)
        assert torch.all((lse[b, j].double() - l).abs() <= 2.0 ** -11 + slack + 2.0 ** -20 * l.abs()), (b, j)


@pytest.mark.parametrize("tokens, counts", [(3, None), (5, None), (16, None), (64, None), (9, [9, 4, 1, 9, 0, 7, 5])])
def test_neighbours_keep_their_bits(gpu_lib, tokens, counts):
    """Whole and split requests, a far one and one with a NaN among them."""
    import torch
    seqs = [30000, 300, 70000, 0, 5000, 9, 2048]
    build = lambda: Case(seqs, WIDE, tokens, counts=counts, seed=tokens)  # noqa: E731
    plain = build()
    base = run(gpu_lib, plain)
    one, two = build(), build()
    far(one, 2)
    got = run(gpu_lib, one)
    same(one, got, base, [b for b in range(7) if b != 2])
    check_far(one, *got, 2)
    far(two, 2)
    nan(two, 5)
    both = run(gpu_lib, two)
    same(two, both, base, [0, 1, 3, 4, 6])
    same(two, both, got, [2])                   # its own bits do not depend on which others are done again
    bad = torch.zeros(tokens, 64, dtype=torch.bool, device="cuda")
    bad[0, 3] = True
    n = two.drafted(5)
    assert torch.equal(torch.isnan(both[1][5, :n]), bad[:n]) and torch.equal(torch.isnan(both[0][5, :n]).any(-1), bad[:n])


@pytest.mark.parametrize("batch, tokens, context", [(300, 5, 1 << 14), (1024, 3, 1 << 12), (100, 16, 512), (200, 6, 768)])
def test_neighbours_in_large_batches(gpu_lib, batch, tokens, context):
    """More requests than ranges (merged by cuts), and tables too short for a merge: every third request far."""
    rng = np.random.default_rng(batch)
    seqs = np.exp(rng.uniform(0, np.log(min(context, 3000)), size=batch)).astype(int).tolist()
    seqs[batch // 2] = context
    plain, case = Case(seqs, context, tokens, seed=batch), Case(seqs, context, tokens, seed=batch)
    base = run(gpu_lib, plain)
    again = [b for b in range(batch) if b % 3 == 1 and seqs[b] > 512]
    for b in again:
        far(case, b)
    got = run(gpu_lib, case)
    same(case, got, base, [b for b in range(batch) if b not in again])
    for b in again[:20]:
        check_far(case, *got, b)


@pytest.mark.parametrize("context", [WIDE, 768])
def test_nothing_stays_behind(gpu_lib, context):
    """One workspace and one graph, with requests done again and without: the same bits as fresh calls, and the rest
    of the workspace's header is zero after each."""
    import torch
    B, T = (4, 6) if context == WIDE else (160, 6)
    seqs = [min(s, context) for s in [40000, 700, 3, 9000]] * (B // 4)
    plain, case = Case(seqs, context, T, seed=3), Case(seqs, context, T, seed=3)
    nan(case, 1)
    far(case, 3)
    want = [run(gpu_lib, plain), run(gpu_lib, case)]
    ws = gpu_lib.new_tree_workspace(B, T)
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    q, draft = plain.q.clone(), plain.draft.clone()
    live = Case(seqs, context, T, seed=3)
    gpu_lib.dsa_mla_tree_decode(*live.args(), out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu_lib.dsa_mla_tree_decode(*live.args(), out=out, lse=lse, workspace=ws)
    for turn in (0, 1, 1, 0, 1, 0):
        live.q.copy_(case.q if turn else q)
        live.draft.copy_(case.draft if turn else draft)
        out.zero_()
        lse.zero_()
        graph.replay()
        same(live, (out, lse), want[turn], range(B))
        assert not ws[:256].any()
    assert gpu_lib.get_error(ws) == 0
