"""GPU tests of dsa_mla_tree_decode's kernel on clusters of two CTAs: two drafted tokens, tables that are wide (a
large max_context), whatever the requests' lengths.  Cases, fp64 reference and tolerances as in test_gpu_mla_tree.py."""
import numpy as np
import pytest

from test_gpu_mla_tree import Case, run
from test_gpu_mla_tree_long import check_large_scores

pytestmark = pytest.mark.gpu

WIDE = 1 << 19   # one request is enough for this kernel


@pytest.mark.parametrize("seq", [0, 1, 4, 5, 60, 61, 64, 65, 68, 252, 255, 256, 257, 260, 300, 508, 512, 513, 516, 768, 1000,
                                 2048, 2049, 70000])
def test_two_one_request(gpu_lib, seq):
    case = Case([seq], WIDE, 2, seed=seq)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("batch", [2, 7, 75, 76, 77, 152, 300, 1024])
def test_two_batches(gpu_lib, batch):
    rng = np.random.default_rng(batch)
    seqs = np.exp(rng.uniform(0, np.log(40000 if batch <= 7 else 3000), size=batch)).astype(int)
    seqs[rng.integers(batch, size=2)] = 0
    case = Case(seqs.tolist(), WIDE if batch <= 77 else 1 << 14, 2, seed=batch)
    case.check(*run(gpu_lib, case), rows=None if batch <= 77 else rng.choice(batch, 100, replace=False).tolist())


@pytest.mark.parametrize("batch, context", [(600, 768), (1024, 1024), (150, 2048)])
def test_two_narrow_tables(gpu_lib, batch, context):
    """Batches whose requests are never split, and others of a few blocks."""
    rng = np.random.default_rng(batch)
    case = Case(rng.integers(0, context + 1, batch).tolist(), context, 2, seed=batch)
    case.check(*run(gpu_lib, case), rows=rng.choice(batch, 100, replace=False).tolist())


def test_two_counts(gpu_lib):
    """Padding holds NaN, is not seen and not written."""
    seqs = [0, 5, 700, 8192, 1, 20000, 64, 300, 2000]
    counts = [0, 2, 1, 1, 0, 2, 1, 1, 2]
    case = Case(seqs, WIDE, 2, counts=counts, masks=[[3, 3]] * 9, seed=1)
    for b, c in enumerate(counts):
        case.draft[b, c:] = float("nan")
        case.q[b, c:] = float("nan")
    case.check(*run(gpu_lib, case), untouched=7.0)
    case = Case([100, 30000], WIDE, 2, counts=[0, 0], seed=5)
    case.check(*run(gpu_lib, case), untouched=7.0)


def test_two_masks(gpu_lib):
    masks = [[0, 0], [3, 3], [2, 1], [1 << 63 | 1 << 40, 3], [0, 0], [0, 2]]
    case = Case([100, 1000, 0, 257, 0, 0], WIDE, 2, masks=masks, seed=3)
    case.check(*run(gpu_lib, case))


def test_two_unseen_entries_are_never_used(gpu_lib):
    """NaN behind the live entries, in pages of no request, in drafted entries that nobody sees."""
    import torch
    case = Case([5, 70, 257, 0, 1030, 20005], WIDE, 2, masks=[[1, 1]] * 6, seed=4)
    case.draft[:, 1] = float("nan")
    live = torch.zeros(case.kv.shape[:2], dtype=torch.bool)
    for b, s in enumerate(case.seqs):
        for t in range(-(-s // 4)):
            live[case.table[b, t // 64], t % 64] = True
    case.kv[~live.cuda()] = float("nan")
    case.check(*run(gpu_lib, case))


def test_two_rising_scores(gpu_lib):
    """Scores that grow along a request, by far more than a weight's range, and the drafted ones alone."""
    case = Case([6000, 3000, 20000, 0], WIDE, 2, seed=5, scale=1.0 / 24.0)
    n = -(-6000 // 256)
    for i in range(n):
        case.kv[case.table[0, i].long()] *= 4.0 ** (i * 6 / n - 3)
    case.draft[2, 1] *= 512.0
    out, lse = run(gpu_lib, case)
    check_large_scores(case, out, lse, range(4))


def test_two_scores_far_below_zero(gpu_lib):
    """The first block has no good page, and every score is hundreds below zero."""
    import torch
    case = Case([40000], WIDE, 2, masks=[[0, 0]], seed=7, scale=1.0)
    direction = torch.randn(576, generator=torch.Generator().manual_seed(1)).cuda()
    case.q[:] = direction.to(torch.bfloat16)
    case.kv[:] = (-direction + 0.05 * torch.randn(case.kv.shape, generator=torch.Generator().manual_seed(2)).cuda()).to(torch.bfloat16)
    table = case.table.clone()
    case.table[0, :2] = -1
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_BAD_PAGE)
    t = torch.arange(128, 10000, device="cuda")
    kv = case.kv[table[0].long()[t // 64], t % 64].double()
    for j in range(2):
        s = case.q[0, j].double() @ kv.T
        slack = float((case.q[0, j].double().abs() @ kv.abs().T).max()) * 2.0 ** -21
        l = torch.logsumexp(s, 1)
        assert float(l.max()) < -300
        assert torch.all((lse[0, j].double() - l).abs() <= 2.0 ** -11 + slack + 2.0 ** -20 * l.abs())
        w = torch.softmax(s, 1)
        o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
        assert not ((out[0, j].double() - o).abs() > (2.0 ** -8 + 2.0 ** -10 + 2 * slack) * a + 2.0 ** -8 * o.abs()).any()


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_two_zero_and_negative_scale(gpu_lib, scale):
    case = Case([300, 2000, 0], WIDE, 2, seed=6, scale=scale)
    case.check(*run(gpu_lib, case))


def test_two_nan_score(gpu_lib):
    """A query that is NaN or infinite makes its own head's outputs NaN, split or not, and nobody else's."""
    import torch
    case = Case([300, 60000, 5000], WIDE, 2, seed=7)
    case.q[0, 1, 5, 0] = float("nan")
    case.q[1, 0, 63, 575] = float("nan")
    case.q[2, 1, 0, 3] = float("inf")
    out, lse = run(gpu_lib, case)
    bad = torch.zeros(3, 2, 64, dtype=torch.bool, device="cuda")
    bad[0, 1, 5] = bad[1, 0, 63] = bad[2, 1, 0] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(out).any(-1), bad)
    assert torch.equal(torch.isnan(out).all(-1), bad)


def test_two_bad_pages_and_lengths(gpu_lib):
    """Live page ids outside the pool (of either page of a block, of both) are left out and flagged."""
    import torch
    case = Case([2000, 700, 20000], WIDE, 2, seed=9)
    table = case.table.clone()
    bad = {0: [2], 1: [0, 1], 2: [15, 40, 41, 77]}
    for b, pages in bad.items():
        for i in pages:
            case.table[b, i] = case.kv.shape[0] if i % 2 else -7
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_BAD_PAGE)
    for b, pages in bad.items():
        for j in range(2):
            t = torch.arange(-(-case.seqs[b] // 4), device="cuda")
            for i in pages:
                t = t[t // 64 != i]
            own = [i for i in range(2) if case.masks[b][j] >> i & 1]
            kv = torch.cat([case.kv[table[b].long()[t // 64], t % 64], case.draft[b, own]]).double()
            s = case.scale * (case.q[b, j].double() @ kv.T)
            w = torch.softmax(s, dim=1)
            o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
            assert not ((out[b, j].double() - o).abs() > (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * o.abs() + 1e-12).any()
    case = Case([WIDE + 5000, -3, 300], WIDE, 2, counts=[9, -1, 2], seed=10)
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_SEQ_LEN_CLAMPED | gpu_lib.DEVERR_BAD_RANGE)
    case.check(out, lse, untouched=7.0)


def test_two_offsets(gpu_lib):
    """Tensors off 32-byte boundaries (16 is what is asked for)."""
    import torch
    case = Case([5000, 300], WIDE, 2, seed=11)
    off = lambda t, pad: torch.cat([t.new_zeros(pad), t.flatten()])[pad:].view(t.shape)  # noqa: E731
    case.q, case.draft, case.kv = off(case.q, 8), off(case.draft, 8), off(case.kv, 8)
    out = torch.zeros(2 * 2 * 64 * 512 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(2, 2, 64, 512)
    lse = torch.zeros(2 * 2 * 64 + 1, device="cuda")[1:].view(2, 2, 64)
    case.check(*run(gpu_lib, case, out=out, lse=lse))


def test_two_same_bits(gpu_lib):
    """Same arguments, same bits: again and again, replayed, and the replay takes new lengths; two streams at once."""
    import torch
    case = Case([30000, 900, 0, 65536], WIDE, 2, seed=12)
    ws = gpu_lib.new_tree_workspace(4, 2)
    first = [t.clone() for t in gpu_lib.dsa_mla_tree_decode(*case.args(), workspace=ws)]
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu_lib.dsa_mla_tree_decode(*case.args(), out=out, lse=lse, workspace=ws)
    other, out2, lse2 = gpu_lib.new_tree_workspace(4, 2), torch.empty_like(out), torch.empty_like(lse)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        out.zero_()
        lse.zero_()
        with torch.cuda.stream(stream):
            gpu_lib.dsa_mla_tree_decode(*case.args(), out=out2, lse=lse2, workspace=other)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in [(out, first[0]), (lse, first[1]), (out2, first[0]), (lse2, first[1])]:
            assert torch.equal(a, b)
    case.seqs = [17, 65536, 4000, 0]
    case.seq.copy_(torch.tensor(case.seqs, dtype=torch.int32))
    case.table.copy_(torch.randint(case.kv.shape[0], case.table.shape, dtype=torch.int32).cuda())
    graph.replay()
    case.check(out, lse)
    assert gpu_lib.get_error(ws) == 0


@pytest.mark.parametrize("seed", range(8))
def test_two_random(gpu_lib, seed):
    rng = np.random.default_rng(2000 + seed)
    batch = int(rng.integers(1, 40))
    seqs = np.exp(rng.uniform(0, np.log(9000 if batch > 8 else 60000), batch)).astype(int).tolist()
    counts = rng.integers(0, 3, batch).tolist() if seed % 2 else None
    case = Case(seqs, 1 << int(rng.integers(18, 21)), 2, counts=counts, seed=seed, q_mag=float(rng.uniform(0.1, 3)),
                masks=[rng.integers(0, 4, 2).tolist() for _ in seqs])
    case.check(*run(gpu_lib, case), untouched=7.0)
