"""GPU tests of dsa_mla_tree_decode against the same attention in fp64.

Tolerances from the arithmetic, as for dsa_mla_decode.  Scores: 576 exact bf16 products summed in
fp32 by the tensor cores; with |s| below 40 (log2 units) their error is under 2^-12, so a weight's
is, relatively.  Each weight is rounded to bf16 for the second product (half a step: 2^-8 of it)
while the sum that divides it is not, so |o - o_ref| <= (2^-8 + 2^-10) o_abs, o_abs = sum_t w_t |v_t|,
before o itself is rounded to bf16 (2^-8 |o|).  lse: the sum of fp32 weights, each within 2^-12
relatively: |lse - lse_ref| <= 2^-11 + 2^-20 |lse|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SCALE = 192.0 ** -0.5


def tree(rng, tokens, back=4):
    """Masks of a random tree: each token sees its ancestors and itself."""
    seen = []
    for j in range(tokens):
        parent = int(rng.integers(max(-1, j - back), j))
        seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
    return seen


class Case:
    """q, cache, table, lengths, drafted entries and masks on the GPU; live pages scattered over the pool."""

    def __init__(self, seqs, max_context, tokens, counts=None, masks=None, seed=1, spare=3, scale=SCALE, q_mag=1.0):
        import torch
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(seqs)
        self.seqs, self.max_context, self.tokens, self.counts, self.scale = list(seqs), max_context, tokens, counts, scale
        self.masks = masks or [tree(rng, tokens) for _ in seqs]
        pages = [-(-min(max(s, 0), max_context) // 256) for s in self.seqs]
        total = sum(pages) + spare
        perm = torch.randperm(total, generator=g).to(torch.int32)
        table = torch.full((B, max_context // 256), -1, dtype=torch.int32)
        at = 0
        for b, p in enumerate(pages):
            table[b, :p] = perm[at:at + p]
            at += p
        self.table = table.cuda()
        self.seq = torch.tensor(self.seqs, dtype=torch.int32).cuda()
        self.kv = torch.randn(total, 64, 576, generator=g).to(torch.bfloat16).cuda()
        self.draft = torch.randn(B, tokens, 576, generator=g).to(torch.bfloat16).cuda()
        self.q = (torch.randn(B, tokens, 64, 576, generator=g) * q_mag).to(torch.bfloat16).cuda()
        words = [[m - (1 << 64) if m >> 63 else m for m in row] for row in self.masks]
        self.mask = torch.tensor(words, dtype=torch.int64).cuda()
        self.count = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()

    def args(self):
        return self.q, self.kv, self.table, self.seq, self.max_context, self.draft, self.mask, self.scale

    def drafted(self, b):
        return self.tokens if self.counts is None else min(max(self.counts[b], 0), self.tokens)

    def entries(self, b, j):
        """What token j of request b sees, in fp64."""
        import torch
        n = -(-min(max(self.seqs[b], 0), self.max_context) // 4)
        t = torch.arange(n, device="cuda")
        kv = self.kv[self.table[b].long()[t // 64], t % 64]
        own = [i for i in range(self.drafted(b)) if self.masks[b][j] >> i & 1]
        return torch.cat([kv, self.draft[b, own]]).double()

    def check(self, out, lse, rows=None, untouched=None):
        import torch
        for b in range(len(self.seqs)) if rows is None else rows:
            for j in range(self.tokens):
                if j >= self.drafted(b):
                    if untouched is not None:
                        assert torch.all(out[b, j] == untouched) and torch.all(lse[b, j] == untouched), (b, j)
                    continue
                kv = self.entries(b, j)
                if len(kv) == 0:
                    assert not out[b, j].any() and torch.all(torch.isneginf(lse[b, j])), (b, j)
                    continue
                s = self.scale * (self.q[b, j].double() @ kv.T)
                w = torch.softmax(s, dim=1)
                o, a, l = w @ kv[:, :512], w @ kv[:, :512].abs(), torch.logsumexp(s, 1)
                err = (out[b, j].double() - o).abs()
                tol = (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * o.abs() + 1e-12
                assert not (err > tol).any(), f"request {b} token {j}: out off by {float((err / a).max())} of o_abs"
                dl = (lse[b, j].double() - l).abs()
                assert torch.all(dl <= 2.0 ** -11 + 2.0 ** -20 * l.abs()), f"request {b} token {j}: lse {float(dl.max())}"


def run(lib, case, error=0, **kw):
    import torch
    ws = lib.new_tree_workspace(len(case.seqs), case.tokens)
    out = torch.full((len(case.seqs), case.tokens, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((len(case.seqs), case.tokens, 64), 7.0, device="cuda")
    kw = dict(dict(token_counts=case.count, out=out, lse=lse, workspace=ws), **kw)
    out, lse = lib.dsa_mla_tree_decode(*case.args(), **kw)
    assert lib.get_error(ws) == error
    return out, lse


@pytest.mark.parametrize("seq", [0, 1, 4, 5, 60, 61, 64, 65, 255, 256, 257, 260, 300, 512, 513, 1000, 2048])
def test_tree_one_request(gpu_lib, seq):
    """One request: drafted entries alone, beside a partial page, behind whole pages, in either half of a block."""
    case = Case([seq], 2048, 5, seed=seq + 1)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 7, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64])
def test_tree_tokens(gpu_lib, tokens):
    """Every size of a tree's last 16-entry step, odd last tokens; long and short requests and an empty one."""
    case = Case([0, 3, 257, 1024, 4321, 300], 8192, tokens, seed=10 + tokens)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("batch", [1, 2, 7, 64, 75, 76, 77, 152, 300, 1024])
def test_tree_batches(gpu_lib, batch):
    rng = np.random.default_rng(batch)
    hi = 40000 if batch <= 7 else 4096
    seqs = np.exp(rng.uniform(0, np.log(hi), size=batch)).astype(int)
    seqs[rng.integers(batch)] = hi
    if batch > 3:
        seqs[rng.integers(batch, size=2)] = 0
    tokens = 6 if batch <= 152 else 3
    case = Case(seqs.tolist(), 40960 if batch <= 7 else 4096, tokens, seed=batch)
    case.check(*run(gpu_lib, case), rows=None if batch <= 152 else rng.choice(batch, 100, replace=False).tolist())


@pytest.mark.parametrize("tokens", [1, 2, 9, 64])
def test_tree_long_requests(gpu_lib, tokens):
    """Requests over many ranges, joined by the merge, beside short ones."""
    case = Case([300, 100000, 7, 0, 5000, 262145], 1 << 19, tokens, seed=tokens)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("tokens, seed", [(2, 0), (5, 1), (16, 2), (27, 3), (64, 4)])
def test_tree_counts(gpu_lib, tokens, seed):
    """Trees of different sizes in one batch: padding is neither seen (its entries hold NaN) nor written."""
    rng = np.random.default_rng(seed)
    seqs = [0, 5, 700, 8192, 1, 20000, 64, 300]
    counts = [0, tokens, 1, tokens // 2, 0, tokens, max(tokens - 1, 0), 1]
    masks = [[int(rng.integers(1 << 62)) | 1 << j for j in range(tokens)] for _ in seqs]  # bits past the counts too
    case = Case(seqs, 20480, tokens, counts=counts, masks=masks, seed=seed)
    for b, c in enumerate(counts):
        case.draft[b, c:] = float("nan")
        case.q[b, c:] = float("nan")
    case.check(*run(gpu_lib, case), untouched=7.0)


def test_tree_masks(gpu_lib):
    """No drafted entry, all of them, one other only, none of an empty request's (a row without entries)."""
    T = 20
    full = (1 << T) - 1
    masks = [[0] * T, [full] * T, [1 << (T - 1 - j) for j in range(T)], [(1 << 63 | 1 << 40) + full - (1 << j) for j in range(T)],
             [0] * T, [0 if j % 2 else 1 << j for j in range(T)]]
    case = Case([100, 1000, 0, 257, 0, 0], 1024, T, masks=masks, seed=3)
    case.check(*run(gpu_lib, case))


def test_tree_unseen_entries_are_never_used(gpu_lib):
    """NaN and infinities behind the live entries, in pages of no request, in drafted entries that nobody sees."""
    case = Case([5, 70, 257, 0, 1030], 2048, 11, seed=4)
    unseen = [3, 9]
    for b in range(5):
        case.masks[b] = [m & ~sum(1 << i for i in unseen) for m in case.masks[b]]
        case.draft[b, unseen[0]] = float("nan")
        case.draft[b, unseen[1]] = float("inf")
    import torch
    case.mask = torch.tensor(case.masks, dtype=torch.int64).cuda()
    live = torch.zeros(case.kv.shape[:2], dtype=torch.bool)
    for b, s in enumerate(case.seqs):
        for t in range(-(-s // 4)):
            live[case.table[b, t // 64], t % 64] = True
    case.kv[~live.cuda()] = float("nan")
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("tokens", [2, 7])
def test_tree_running_max(gpu_lib, tokens):
    """Pages whose keys grow by 4x along a request: the running maximum is raised over a filled accumulator,
    by the cache's pages and by the drafted ones."""
    case = Case([6000, 3000, 40000], 40960, tokens, seed=5, scale=1.0 / 24.0)
    for b in range(3):
        n = -(-case.seqs[b] // 256)
        for i in range(n):
            case.kv[case.table[b, i].long()] *= 4.0 ** (i * 6 / n - 3)
    case.draft *= 64.0
    out, lse = run(gpu_lib, case)
    import torch
    for b in range(3):
        for j in range(tokens):
            kv = case.entries(b, j)
            s = case.scale * (case.q[b, j].double() @ kv.T)
            # scores of thousands: fp32 sums of 576 products are off by 2^-21 of |s|'s terms at most
            size = case.scale * (case.q[b, j].double().abs() @ kv.abs().T)
            slack = float((size * 2.0 ** -21).max())
            w = torch.softmax(s, dim=1)
            o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
            tol = (2.0 ** -8 + 2.0 ** -10 + 2 * slack) * a + 2.0 ** -8 * o.abs() + 1e-12
            assert not ((out[b, j].double() - o).abs() > tol).any(), (b, j)
            l = torch.logsumexp(s, 1)
            assert torch.all((lse[b, j].double() - l).abs() <= 2.0 ** -11 + slack + 2.0 ** -20 * l.abs()), (b, j)


def test_tree_zero_and_negative_scale(gpu_lib):
    for scale in (0.0, -0.05):
        case = Case([300, 2000], 2048, 3, seed=6, scale=scale)
        case.check(*run(gpu_lib, case))


def test_tree_nan_score(gpu_lib):
    """A query that is NaN makes its own head's outputs NaN, split or not, and nobody else's."""
    import torch
    case = Case([300, 60000], 1 << 16, 4, seed=7)
    case.q[0, 1, 5, 0] = float("nan")
    case.q[1, 2, 63, 575] = float("nan")
    out, lse = run(gpu_lib, case)
    bad = torch.zeros(2, 4, 64, dtype=torch.bool, device="cuda")
    bad[0, 1, 5] = bad[1, 2, 63] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(out).all(-1), bad)
    assert torch.equal(torch.isnan(out).any(-1), bad)


def test_tree_chain_equals_next_n(gpu_lib):
    """A chain of drafted tokens whose entries are in the cache already, one a C4 entry: what dsa_mla_decode
    gives for the token that sees them all."""
    import torch
    case = Case([1000, 4000], 4096, 1, seed=8)
    case.masks = [[1], [1]]
    ws = gpu_lib.new_mla_workspace(2, 1)
    # the last entry of each request moves out of the cache into the draft
    shorter = [s - 4 for s in case.seqs]
    for b, s in enumerate(case.seqs):
        t = -(-s // 4) - 1
        case.draft[b, 0] = case.kv[case.table[b, t // 64].long(), t % 64]
    want, want_lse = gpu_lib.dsa_mla_decode(case.q[:, 0].contiguous(), case.kv, case.table, case.seq, 4096, SCALE,
                                            workspace=ws)
    seq = torch.tensor(shorter, dtype=torch.int32).cuda()
    out, lse = gpu_lib.dsa_mla_tree_decode(case.q, case.kv, case.table, seq, 4096, case.draft, case.mask, SCALE)
    assert torch.all((lse[:, 0] - want_lse).abs() <= 2.0 ** -10 + 2.0 ** -19 * want_lse.abs())
    assert torch.all((out[:, 0].float() - want.float()).abs() <= 2.0 ** -6)


def test_tree_bad_page_and_lengths(gpu_lib):
    """A live page id outside the pool is left out and flagged; lengths and counts out of range are held."""
    import torch
    case = Case([2000, 700, 4000], 4096, 4, seed=9)
    table = case.table.clone()
    case.table[0, 2], case.table[2, 15] = case.kv.shape[0], -7
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_BAD_PAGE)
    for b, bad in ((0, 2), (2, 15)):
        for j in range(4):
            n = -(-case.seqs[b] // 4)
            t = torch.arange(n, device="cuda")
            t = t[t // 64 != bad]
            own = [i for i in range(4) if case.masks[b][j] >> i & 1]
            kv = torch.cat([case.kv[table[b].long()[t // 64], t % 64], case.draft[b, own]]).double()
            s = SCALE * (case.q[b, j].double() @ kv.T)
            w = torch.softmax(s, dim=1)
            o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
            assert not ((out[b, j].double() - o).abs() > (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * o.abs() + 1e-12).any()
    case = Case([5000, -3, 300], 4096, 3, counts=[9, -1, 2], seed=10)
    out, lse = run(gpu_lib, case, error=gpu_lib.DEVERR_SEQ_LEN_CLAMPED | gpu_lib.DEVERR_BAD_RANGE)
    case.check(out, lse, untouched=7.0)


def test_tree_same_bits(gpu_lib):
    """Same arguments, same bits: with one workspace again and again, eager and replayed, after other calls."""
    import torch
    case = Case([30000, 900, 0, 65536], 1 << 16, 9, seed=11)
    other = Case([700, 20000, 3, 1], 1 << 16, 9, seed=12)
    ws = gpu_lib.new_tree_workspace(4, 9)
    first = [t.clone() for t in gpu_lib.dsa_mla_tree_decode(*case.args(), workspace=ws)]
    gpu_lib.dsa_mla_tree_decode(*other.args(), workspace=ws)
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu_lib.dsa_mla_tree_decode(*case.args(), out=out, lse=lse, workspace=ws)
    for _ in range(3):
        out.zero_()
        lse.zero_()
        graph.replay()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # other contents, the same graph
    case.seq.copy_(torch.tensor([17, 65536, 4000, 0], dtype=torch.int32))
    case.table.copy_(torch.randint(case.kv.shape[0], case.table.shape, dtype=torch.int32).cuda())
    case.seqs = [17, 65536, 4000, 0]
    graph.replay()
    case.check(out, lse)
    assert gpu_lib.get_error(ws) == 0


def test_tree_streams(gpu_lib):
    """Calls on two streams at a time, a workspace each, one of them not the tensors' own stream."""
    import torch
    cases = [Case([40000, 100], 40960, 8, seed=13), Case([9000, 33000], 40960, 5, seed=14)]
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
