"""GPU tests of dsa_mla_tree_decode's kernel on clusters of four CTAs: calls whose table is wide (a large
max_context), whatever the requests' lengths, for trees of more than two tokens.  Cases, fp64 reference and
tolerances as in test_gpu_mla_tree.py."""
import numpy as np
import pytest

from test_gpu_mla_tree import Case, run, tree

pytestmark = pytest.mark.gpu

WIDE = 1 << 18   # 3 tokens of one request are enough for this kernel


@pytest.mark.parametrize("seq", [0, 1, 4, 5, 60, 61, 64, 65, 68, 252, 255, 256, 257, 260, 300, 508, 512, 513, 516, 768, 1000,
                                 2048, 2049, 70000])
@pytest.mark.parametrize("tokens", [3, 5])
def test_long_one_request(gpu_lib, seq, tokens):
    """Drafted entries in either half of a block, behind partial and whole pages, alone; split and unsplit."""
    case = Case([seq], WIDE, tokens, seed=seq + tokens)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("tokens", [3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64])
def test_long_tokens(gpu_lib, tokens):
    """Tiles of one to four tokens at the end; long and short requests, an empty one, more than a round."""
    case = Case([0, 3, 257, 1024, 4321, 300, 30000], WIDE, tokens, seed=10 + tokens)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("batch", [2, 7, 35, 36, 37, 72, 300, 1024])
def test_long_batches(gpu_lib, batch):
    rng = np.random.default_rng(batch)
    seqs = np.exp(rng.uniform(0, np.log(40000 if batch <= 7 else 3000), size=batch)).astype(int)
    seqs[rng.integers(batch, size=2)] = 0
    case = Case(seqs.tolist(), WIDE if batch <= 72 else 1 << 14, 5, seed=batch)
    case.check(*run(gpu_lib, case), rows=None if batch <= 72 else rng.choice(batch, 100, replace=False).tolist())


@pytest.mark.parametrize("tokens, seed", [(3, 1), (10, 2), (27, 3), (64, 4)])
def test_long_counts(gpu_lib, tokens, seed):
    """Padded trees, whole tiles of padding among them: padding holds NaN, is not seen and not written."""
    rng = np.random.default_rng(seed)
    seqs = [0, 5, 700, 8192, 1, 20000, 64, 300, 2000]
    counts = [0, tokens, 1, tokens // 2, 0, tokens, max(tokens - 1, 0), 1, 2]
    masks = [[int(rng.integers(1 << 62)) | 1 << j for j in range(tokens)] for _ in seqs]
    case = Case(seqs, WIDE, tokens, counts=counts, masks=masks, seed=seed)
    for b, c in enumerate(counts):
        case.draft[b, c:] = float("nan")
        case.q[b, c:] = float("nan")
    case.check(*run(gpu_lib, case), untouched=7.0)


def test_long_all_padding(gpu_lib):
    case = Case([100, 30000], WIDE, 9, counts=[0, 0], seed=5)
    case.check(*run(gpu_lib, case), untouched=7.0)


def test_long_masks(gpu_lib):
    """No drafted entry, all of them, one other only, none of an empty request's (rows without entries)."""
    T = 20
    full = (1 << T) - 1
    masks = [[0] * T, [full] * T, [1 << (T - 1 - j) for j in range(T)], [(1 << 63 | 1 << 40) + full - (1 << j) for j in range(T)],
             [0] * T, [0 if j % 2 else 1 << j for j in range(T)]]
    case = Case([100, 1000, 0, 257, 0, 0], WIDE, T, masks=masks, seed=3)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("tokens", [3, 11, 64])
def test_long_unseen_entries_are_never_used(gpu_lib, tokens):
    """NaN and infinities behind the live entries, in pages of no request, in drafted entries that nobody sees."""
    import torch
    case = Case([5, 70, 257, 0, 1030, 20005], WIDE, tokens, seed=4)
    unseen = [1, tokens - 1]
    for b in range(len(case.seqs)):
        case.masks[b] = [m & ~sum(1 << i for i in unseen) for m in case.masks[b]]
        case.draft[b, unseen[0]] = float("nan")
        case.draft[b, unseen[1]] = float("inf")
    words = [[m - (1 << 64) if m >> 63 else m for m in row] for row in case.masks]
    case.mask = torch.tensor(words, dtype=torch.int64).cuda()
    live = torch.zeros(case.kv.shape[:2], dtype=torch.bool)
    for b, s in enumerate(case.seqs):
        for t in range(-(-s // 4)):
            live[case.table[b, t // 64], t % 64] = True
    case.kv[~live.cuda()] = float("nan")
    case.check(*run(gpu_lib, case))


def check_large_scores(case, out, lse, requests):
    """Scores of hundreds or thousands: fp32 sums of 576 products are off by 2^-21 of the sum of their sizes."""
    import torch
    for b in requests:
        for j in range(case.tokens):
            kv = case.entries(b, j)
            s = case.scale * (case.q[b, j].double() @ kv.T)
            slack = float((case.scale * (case.q[b, j].double().abs() @ kv.abs().T)).max()) * 2.0 ** -21
            w = torch.softmax(s, dim=1)
            o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
            tol = (2.0 ** -8 + 2.0 ** -10 + 2 * slack) * a + 2.0 ** -8 * o.abs() + 1e-12
            assert not ((out[b, j].double() - o).abs() > tol).any(), (b, j)
            l = torch.logsumexp(s, 1)
            assert torch.all((lse[b, j].double() - l).abs() <= 2.0 ** -11 + slack + 2.0 ** -20 * l.abs()), (b, j)


@pytest.mark.parametrize("tokens", [3, 6])
def test_long_scores_far_above_the_first(gpu_lib, tokens):
    """A request whose later scores pass the first block's by more than its reference reaches (its sums overflow):
    the call is done again, its neighbours' rows with it."""
    case = Case([6000, 3000, 20000, 0], WIDE, tokens, seed=5, scale=1.0 / 24.0)
    for i in range(24):
        case.kv[case.table[1, i % 12].long()] *= 4.0 if i < 12 else 1.0
    n = -(-6000 // 256)
    for i in range(n):
        case.kv[case.table[0, i].long()] *= 4.0 ** (i * 6 / n - 3)
    out, lse = run(gpu_lib, case)
    check_large_scores(case, out, lse, range(4))


def test_long_drafts_far_above_the_cache(gpu_lib):
    """Only the drafted entries' scores pass the reference, of one token of one request among many."""
    case = Case([700] * 20, 1 << 15, 4, seed=6, scale=1.0 / 24.0)
    case.draft[13, 2] *= 512.0
    out, lse = run(gpu_lib, case)
    check_large_scores(case, out, lse, range(20))


@pytest.mark.parametrize("length", [520, 40000])
def test_long_scores_far_below_zero(gpu_lib, length):
    """The first block has no good page, so no reference, and every score is hundreds below zero."""
    import torch
    case = Case([length], WIDE, 3, masks=[[0, 0, 0]], seed=7, scale=1.0)
    direction = torch.randn(576, generator=torch.Generator().manual_seed(1)).cuda()
    case.q[:] = (direction * 1.0).to(torch.bfloat16)
    case.kv[:] = (-direction + 0.05 * torch.randn(case.kv.shape, generator=torch.Generator().manual_seed(2)).cuda()).to(torch.bfloat16)
    table = case.table.clone()
    case.table[0, :2] = -1
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_BAD_PAGE)
    n = -(-length // 4)
    t = torch.arange(128, n, device="cuda")
    if len(t) == 0:
        return
    kv = case.kv[table[0].long()[t // 64], t % 64].double()
    for j in range(3):
        s = case.q[0, j].double() @ kv.T
        slack = float((case.q[0, j].double().abs() @ kv.abs().T).max()) * 2.0 ** -21
        l = torch.logsumexp(s, 1)
        assert float(l.max()) < -300
        assert torch.all((lse[0, j].double() - l).abs() <= 2.0 ** -11 + slack + 2.0 ** -20 * l.abs())
        w = torch.softmax(s, 1)
        o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
        assert not ((out[0, j].double() - o).abs() > (2.0 ** -8 + 2.0 ** -10 + 2 * slack) * a + 2.0 ** -8 * o.abs()).any()


def test_long_large_values(gpu_lib):
    """Values near bf16's end whose weighted sum is finite."""
    case = Case([900, 20000], WIDE, 3, seed=8, q_mag=2.0 ** -100)
    case.kv[..., :512] *= 2.0 ** 100
    case.draft[..., :512] *= 2.0 ** 100
    case.q[..., 512:] *= 2.0 ** 100
    out, lse = run(gpu_lib, case)
    check_large_scores(case, out, lse, range(2))


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_long_zero_and_negative_scale(gpu_lib, scale):
    case = Case([300, 2000, 0], WIDE, 3, seed=6, scale=scale)
    case.check(*run(gpu_lib, case))


def test_long_nan_score(gpu_lib):
    """A query that is NaN or infinite makes its own head's outputs NaN, split or not, and nobody else's."""
    import torch
    case = Case([300, 60000, 5000], WIDE, 7, seed=7)
    case.q[0, 1, 5, 0] = float("nan")
    case.q[1, 2, 63, 575] = float("nan")
    case.q[2, 6, 0, 3] = float("inf")
    out, lse = run(gpu_lib, case)
    bad = torch.zeros(3, 7, 64, dtype=torch.bool, device="cuda")
    bad[0, 1, 5] = bad[1, 2, 63] = bad[2, 6, 0] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(out).any(-1), bad)
    assert torch.equal(torch.isnan(out).all(-1), bad)


def test_long_bad_pages_and_lengths(gpu_lib):
    """Live page ids outside the pool (in both halves of a block, and a whole block's) are left out and flagged."""
    import torch
    case = Case([2000, 700, 20000], WIDE, 4, seed=9)
    table = case.table.clone()
    bad = {0: [2], 1: [0, 1], 2: [15, 40, 41, 77]}
    for b, pages in bad.items():
        for i in pages:
            case.table[b, i] = case.kv.shape[0] if i % 2 else -7
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_BAD_PAGE)
    for b, pages in bad.items():
        for j in range(4):
            t = torch.arange(-(-case.seqs[b] // 4), device="cuda")
            for i in pages:
                t = t[t // 64 != i]
            own = [i for i in range(4) if case.masks[b][j] >> i & 1]
            kv = torch.cat([case.kv[table[b].long()[t // 64], t % 64], case.draft[b, own]]).double()
            s = case.scale * (case.q[b, j].double() @ kv.T)
            w = torch.softmax(s, dim=1)
            o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
            assert not ((out[b, j].double() - o).abs() > (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * o.abs() + 1e-12).any()
    case = Case([WIDE + 5000, -3, 300], WIDE, 3, counts=[9, -1, 2], seed=10)
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_SEQ_LEN_CLAMPED | gpu_lib.DEVERR_BAD_RANGE)
    case.check(out, lse, untouched=7.0)


def test_long_offsets(gpu_lib):
    """Tensors off 32-byte boundaries (16 is what is asked for)."""
    import torch
    case = Case([5000, 300], WIDE, 5, seed=11)
    off = lambda t, pad: torch.cat([t.new_zeros(pad), t.flatten()])[pad:].view(t.shape)  # noqa: E731
    case.q, case.draft, case.kv = off(case.q, 8), off(case.draft, 8), off(case.kv, 8)
    assert case.q.data_ptr() % 32 == 16
    out = torch.zeros(case.q.shape[0] * 5 * 64 * 512 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(2, 5, 64, 512)
    lse = torch.zeros(2 * 5 * 64 + 1, device="cuda")[1:].view(2, 5, 64)
    case.check(*run(gpu_lib, case, out=out, lse=lse))


def test_long_same_bits(gpu_lib):
    """Same arguments, same bits: again and again, replayed, after a call that was done twice."""
    import torch
    case, other = Case([30000, 900, 0, 65536], WIDE, 9, seed=12), Case([700, 20000, 3, 1], WIDE, 9, seed=13)
    other.draft[1] *= 4096.0
    ws = gpu_lib.new_tree_workspace(4, 9)
    first = [t.clone() for t in gpu_lib.dsa_mla_tree_decode(*case.args(), workspace=ws)]
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu_lib.dsa_mla_tree_decode(*case.args(), out=out, lse=lse, workspace=ws)
    for _ in range(4):
        gpu_lib.dsa_mla_tree_decode(*other.args(), workspace=ws)
        out.zero_()
        lse.zero_()
        graph.replay()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    case.seqs = [17, 65536, 4000, 0]
    case.seq.copy_(torch.tensor(case.seqs, dtype=torch.int32))
    case.table.copy_(torch.randint(case.kv.shape[0], case.table.shape, dtype=torch.int32).cuda())
    graph.replay()
    case.check(out, lse)
    assert gpu_lib.get_error(ws) == 0


def test_long_streams(gpu_lib):
    """Calls on two streams at a time, a workspace each."""
    import torch
    cases = [Case([40000, 100], WIDE, 8, seed=14), Case([9000, 33000], WIDE, 5, seed=15)]
    spaces = [gpu_lib.new_tree_workspace(2, c.tokens) for c in cases]
    outs = [(torch.empty(2, c.tokens, 64, 512, dtype=torch.bfloat16, device="cuda"),
             torch.empty(2, c.tokens, 64, device="cuda")) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, w, (o, l), s in zip(cases, spaces, outs, streams):
            with torch.cuda.stream(s):
                gpu_lib.dsa_mla_tree_decode(*c.args(), out=o, lse=l, workspace=w)
    torch.cuda.synchronize()
    for c, (o, l) in zip(cases, outs):
        c.check(o, l)


def test_long_own_workspace(gpu_lib):
    case = Case([9000, 33000], WIDE, 5, seed=16)
    for _ in range(3):
        case.check(*gpu_lib.dsa_mla_tree_decode(*case.args()))


@pytest.mark.parametrize("seed", range(12))
def test_long_random(gpu_lib, seed):
    """Random batches: lengths, trees, counts, table widths and scales."""
    rng = np.random.default_rng(1000 + seed)
    batch, tokens = int(rng.integers(1, 40)), int(rng.integers(3, 65))
    seqs = np.exp(rng.uniform(0, np.log(9000 if batch > 8 else 60000), batch)).astype(int).tolist()
    counts = rng.integers(0, tokens + 1, batch).tolist() if seed % 2 else None
    case = Case(seqs, 1 << int(rng.integers(16, 19)), tokens, counts=counts, seed=seed, q_mag=float(rng.uniform(0.1, 3)),
                masks=[tree(rng, tokens, back=int(rng.integers(1, 9))) for _ in seqs])
    case.check(*run(gpu_lib, case), untouched=7.0)
