"""GPU tests of dsa_mla_decode against the same attention in fp64.

Tolerances from the arithmetic.  Scores: 576 exact bf16 products summed in fp32 by the tensor
cores; with |s| below 40 (log2 units) their error is under 2^-12, so a weight's is, relatively.
Each weight is rounded to bf16 for the second product (half a step: 2^-8 of it) while the sum
that divides it is not, so |o - o_ref| <= (2^-8 + 2^-10) * o_abs, o_abs = sum_t w_t |v_t|, before
o itself is rounded to bf16 (2^-8 |o|).  lse: the sum of fp32 weights, each within 2^-12
relatively: |lse - lse_ref| <= 2^-11 + 2^-20 |lse|."""
import numpy as np
import pytest

from sparse_attention_paged_dsa_gb300 import inputs as I

pytestmark = pytest.mark.gpu

SCALE = 192.0 ** -0.5


class Case:
    """q, cache, table and lengths on the GPU; live pages scattered over the pool, the rest -1."""

    def __init__(self, seqs, max_context, next_n=1, seed=1, spare=3, scale=SCALE, q_mag=1.0):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.max_context, self.next_n, self.scale = list(seqs), max_context, next_n, scale
        pages = [-(-(-(-min(max(s, 0), max_context) // 4)) // 64) for s in self.seqs]
        total = sum(pages) + spare
        perm = torch.randperm(total, generator=g).to(torch.int32)
        table = torch.full((len(self.seqs), max_context // 256), -1, dtype=torch.int32)
        at = 0
        for b, p in enumerate(pages):
            table[b, :p] = perm[at:at + p]
            at += p
        self.table = table.cuda()
        self.seq = torch.tensor(self.seqs, dtype=torch.int32).cuda()
        self.kv = torch.randn(total, 64, 576, generator=g).to(torch.bfloat16).cuda()
        self.q = (torch.randn(len(self.seqs), next_n, 64, 576, generator=g) * q_mag).to(torch.bfloat16).cuda()

    def args(self):
        return self.q, self.kv, self.table, self.seq, self.max_context, self.scale

    def live(self, b, j):
        s = min(max(self.seqs[b], 0), self.max_context)
        return -(-max(s - (self.next_n - 1 - j), 0) // 4)

    def reference(self, b, j):
        import torch
        n = self.live(b, j)
        t = torch.arange(n, device="cuda")
        kv = self.kv[self.table[b].long()[t // 64], t % 64].double()
        s = self.scale * (self.q[b, j].double() @ kv.T)
        w = torch.softmax(s, dim=1)
        return w @ kv[:, :512], torch.logsumexp(s, 1), w @ kv[:, :512].abs()

    def check(self, out, lse, rows=None):
        import torch
        out, lse = out.view(len(self.seqs), self.next_n, 64, 512), lse.view(len(self.seqs), self.next_n, 64)
        for b in range(len(self.seqs)) if rows is None else rows:
            for j in range(self.next_n):
                if self.live(b, j) == 0:
                    assert not out[b, j].any() and torch.all(torch.isneginf(lse[b, j])), (b, j)
                    continue
                o, l, a = self.reference(b, j)
                err = (out[b, j].double() - o).abs()
                tol = (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * o.abs() + 1e-12
                assert not (err > tol).any(), f"request {b} token {j}: out off by {float((err / a).max())} of o_abs"
                dl = (lse[b, j].double() - l).abs()
                assert torch.all(dl <= 2.0 ** -11 + 2.0 ** -20 * l.abs()), f"request {b} token {j}: lse {float(dl.max())}"


def run(lib, case, **kw):
    ws = lib.new_mla_workspace(len(case.seqs), case.next_n)
    out, lse = lib.dsa_mla_decode(*case.args(), workspace=ws, **kw)
    assert lib.get_error(ws) == 0
    return out, lse


@pytest.mark.parametrize("seq", [1, 4, 5, 60, 61, 64, 65, 68, 255, 256, 257, 260, 300, 512, 1000, 2048])
def test_decode_one_request(gpu_lib, seq):
    """One request: a single entry, partial 16-entry steps, whole blocks, one entry more."""
    case = Case([seq], 2048, seed=seq)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("next_n", [1, 2, 3, 4])
def test_decode_tokens(gpu_lib, next_n):
    """Each token its own causal length: requests shorter than next_n, and lengths where the
    tokens straddle an entry or a page."""
    case = Case([0, 1, 2, 3, 4, 5, 257, 258, 259, 260, 1024, 1025, 1027, 8192, 4321], 8192, next_n=next_n,
                seed=10 + next_n)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("batch", [1, 2, 7, 64, 151, 152, 153, 300, 1024])
def test_decode_batches(gpu_lib, batch):
    rng = np.random.default_rng(batch)
    hi = 40000 if batch <= 7 else 4096
    seqs = np.exp(rng.uniform(0, np.log(hi), size=batch)).astype(int)
    seqs[rng.integers(batch)] = hi
    if batch > 3:
        seqs[rng.integers(batch, size=2)] = 0
    case = Case(seqs.tolist(), 40960 if batch <= 7 else 4096, seed=batch)
    case.check(*run(gpu_lib, case))


def test_decode_all_empty(gpu_lib):
    case = Case([0, 0, 0], 1024)
    case.check(*run(gpu_lib, case))


def test_decode_one_long_request(gpu_lib):
    """One request of 65,537 entries over every SM, joined by the merge."""
    case = Case([262145], 1 << 19, seed=3)
    case.check(*run(gpu_lib, case))


def test_decode_long_and_short(gpu_lib):
    """A long request among short ones: ranges that hold several requests, a request over many."""
    case = Case([300, 100000, 7, 0, 5000, 1, 70000, 256], 1 << 17, next_n=2, seed=4)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("next_n", [1, 2])
def test_decode_running_max(gpu_lib, next_n):
    """Pages whose keys grow by 4x along a request: the running maximum rises by more than 2^8 again
    and again and the accumulators are rescaled."""
    import torch
    case = Case([6000, 3000], 8192, next_n=next_n, seed=5, scale=1.0 / 24.0)
    for b in range(2):
        n = -(-case.seqs[b] // 256)
        for i in range(n):
            case.kv[case.table[b, i].long()] *= 2.0 ** (i * 4 / n - 2)
    out, lse = run(gpu_lib, case)
    # scores reach about 50 here (72 in log2 units, 2^-17 of them in fp32): the same bounds hold
    case.check(out, lse)
    assert torch.isfinite(out.float()).all()


def test_decode_sharp_softmax(gpu_lib):
    """One dominant entry per head: out is nearly that entry's value row."""
    case = Case([777, 4000], 4096, seed=6, q_mag=1.0, scale=0.02)
    for b in range(2):
        page = case.table[b, 1].long()
        case.kv[page, 13] = case.q[b, 0, 5]
    case.check(*run(gpu_lib, case))


def test_decode_dead_entries_are_never_used(gpu_lib):
    """NaN and infinities behind every live length and on unnamed pages change nothing."""
    import torch
    case = Case([1, 5, 250, 256, 300, 0, 2000], 2048, next_n=2, seed=7)
    want = run(gpu_lib, case)
    used = torch.zeros(case.kv.shape[0], 64, dtype=torch.bool, device="cuda")
    for b in range(len(case.seqs)):
        t = torch.arange(case.live(b, 1), device="cuda")
        used[case.table[b].long()[t // 64], t % 64] = True
    for value in (float("nan"), float("inf"), -3e38):
        case.kv[~used] = value
        got = run(gpu_lib, case)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_entry_only_the_last_token_sees(gpu_lib):
    """An entry past an earlier token's own length may hold anything for that token."""
    import torch
    case = Case([257, 1025], 2048, next_n=2, seed=8)   # token 1 sees one entry more than token 0
    want = run(gpu_lib, case)[0]
    for b, s in enumerate(case.seqs):
        t = case.live(b, 1) - 1
        case.kv[case.table[b, t // 64].long(), t % 64] = float("nan")
    got = run(gpu_lib, case)[0]
    assert torch.equal(got[:, 0], want[:, 0])


def test_decode_shared_pages(gpu_lib):
    """Requests may name the same pages (a shared prefix)."""
    case = Case([2000, 3000, 1000], 4096, seed=9)
    case.table[2, :4] = case.table[0, :4]
    case.table[1, :3] = case.table[0, :3]
    case.check(*run(gpu_lib, case))


def test_decode_bad_pages_and_lengths(gpu_lib):
    """A live page id outside the cache: its entries are left out and the bit is set; a length past
    max_context is held to it, a negative one is 0; the other requests are untouched."""
    import torch
    case = Case([600, 1024, 900, -5, 5000, 100], 1024, seed=11)
    case.table[0, 1] = case.kv.shape[0]
    case.table[2, 0] = -4
    case.table[5, 0] = 1 << 30
    ws = gpu_lib.new_mla_workspace(6)
    out, lse = gpu_lib.dsa_mla_decode(*case.args(), workspace=ws)
    assert gpu_lib.get_error(ws) == gpu_lib.DEVERR_BAD_PAGE | gpu_lib.DEVERR_SEQ_LEN_CLAMPED
    case.check(out, lse, rows=[1, 3, 4])
    assert not out[5].any() and torch.isneginf(lse[5]).all()
    for b, lost in ((0, 1), (2, 0)):
        t = torch.arange(case.live(b, 0), device="cuda")
        t = t[t // 64 != lost]
        kv = case.kv[case.table[b].long()[t // 64], t % 64].double()
        s = case.scale * (case.q[b, 0].double() @ kv.T)
        assert torch.all((torch.logsumexp(s, 1) - lse[b, 0] if lse.dim() == 3 else torch.logsumexp(s, 1) - lse[b]).abs() <= 2.0 ** -10)
        w = torch.softmax(s, 1)
        err = (out.view(6, 64, 512)[b].double() - w @ kv[:, :512]).abs()
        assert not (err > 2.0 ** -6 * (w @ kv[:, :512].abs())).any()


def test_decode_zero_scale_is_the_mean(gpu_lib):
    import torch
    case = Case([3000, 64, 17], 4096, seed=12, scale=0.0)
    out, lse = run(gpu_lib, case)
    case.check(out, lse)
    n = torch.tensor([float(case.live(b, 0)) for b in range(3)])
    assert torch.allclose(lse.view(3, 64)[:, 0].cpu(), n.log(), atol=1e-5)


def test_decode_matches_the_sparse_decode(gpu_lib):
    """On requests of at most 2048 entries: the sparse decode with a full top-k row."""
    import torch
    case = Case([8192, 300, 0, 5000], 8192, seed=13)
    topk = torch.full((4, 2048), -1, dtype=torch.int32)
    for b in range(4):
        topk[b, :case.live(b, 0)] = torch.arange(case.live(b, 0))
    out, lse = run(gpu_lib, case)
    o2, l2 = gpu_lib.dsa_sparse_mla_decode(case.q[:, 0].contiguous(), case.kv, case.table, case.seq, 8192,
                                           topk.cuda(), case.scale)
    assert (out.view(4, 64, 512).float() - o2).abs().max() < 2.0 ** -6
    ok = torch.isfinite(l2)
    assert torch.equal(ok, torch.isfinite(lse.view(4, 64)))
    assert (lse.view(4, 64)[ok] - l2[ok]).abs().max() < 2.0 ** -7


def test_decode_deterministic_and_workspace_reuse(gpu_lib):
    """The same bits on a reused workspace, after another shape's call on it."""
    import torch
    a = Case([9000, 20, 0, 700, 31000], 1 << 15, seed=14)
    b = Case([100] * 9, 512, seed=15)
    ws = gpu_lib.new_mla_workspace(9)
    first = [t.clone() for t in gpu_lib.dsa_mla_decode(*a.args(), workspace=ws)]
    gpu_lib.dsa_mla_decode(*b.args(), workspace=ws)
    again = gpu_lib.dsa_mla_decode(*a.args(), workspace=ws)
    assert gpu_lib.get_error(ws) == 0
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    a.check(*again)


def test_decode_graph_replay_with_other_lengths(gpu_lib):
    """Captured once, replayed with other lengths and page tables: the launch does not depend on them."""
    import torch
    a = Case([8192, 4000, 1, 300], 8192, seed=16, spare=140)
    ws = gpu_lib.new_mla_workspace(4)
    out = torch.empty(4, 1, 64, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, 1, 64, device="cuda")
    gpu_lib.dsa_mla_decode(*a.args(), out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.dsa_mla_decode(*a.args(), out=out, lse=lse, workspace=ws)
    g.replay()
    a.check(out, lse)
    for seqs in ([5, 0, 8000, 8192], [0, 0, 0, 0], [256, 8192, 8192, 8191]):
        a.seqs = seqs
        a.seq.copy_(torch.tensor(seqs, dtype=torch.int32))
        perm = torch.randperm(a.kv.shape[0], device="cuda").to(torch.int32)
        a.table.fill_(-1)
        at = 0
        for b, s in enumerate(seqs):
            n = -(-s // 256)
            a.table[b, :n] = perm[at:at + n]
            at += n
        g.replay()
        torch.cuda.synchronize()
        a.check(out, lse)
    assert gpu_lib.get_error(ws) == 0


def test_decode_two_streams(gpu_lib):
    """Two calls at once on two streams, each with its own workspace."""
    import torch
    cases = [Case([30000, 200], 1 << 15, seed=17), Case([100] * 40, 512, next_n=3, seed=18)]
    want = [run(gpu_lib, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    wss = [gpu_lib.new_mla_workspace(len(c.seqs), c.next_n) for c in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i] = gpu_lib.dsa_mla_decode(*c.args(), workspace=wss[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_decode_refusals(gpu_lib):
    import torch
    c = Case([100], 512, seed=19)
    q, kv, table, seq, ctx, scale = c.args()
    with pytest.raises(ValueError):
        gpu_lib.dsa_mla_decode(q[..., :512], kv, table, seq, ctx, scale)
    with pytest.raises(TypeError):
        gpu_lib.dsa_mla_decode(q.half(), kv, table, seq, ctx, scale)
    with pytest.raises(ValueError):
        gpu_lib.dsa_mla_decode(q, kv, table, seq, 1024, scale)
    with pytest.raises(ValueError):
        gpu_lib.dsa_mla_decode(q, kv.cpu(), table, seq, ctx, scale)
    with pytest.raises(gpu_lib.DsaError):
        gpu_lib.dsa_mla_decode(q, kv, table, seq, ctx, float("inf"))
    with pytest.raises(gpu_lib.DsaError):
        gpu_lib.dsa_mla_decode(q, kv, table, seq, ctx, scale, workspace=torch.zeros(1024, dtype=torch.uint8,
                                                                                    device="cuda"))
    with pytest.raises(gpu_lib.DsaError):
        gpu_lib.dsa_mla_decode(q.expand(1, 5, 64, 576).contiguous(), kv, table, seq, ctx, scale,
                               workspace=gpu_lib.new_mla_workspace(1, 4))
