"""GPU tests of dsa_mla_prefill against the same attention in fp64.

Tolerances from the arithmetic.  Scores: 192 exact bf16 products summed in fp32, below 40 in log2
units here: their error is under 2^-12, so a weight's is, relatively.  Each weight is rounded to
bf16 for the second product (2^-8 of it) while the sum that divides it is not:
|o - o_ref| <= (2^-8 + 2^-10) * o_abs, o_abs = sum_t w_t |v_t|, then o is rounded (2^-8 |o|).
lse: |lse - lse_ref| <= 2^-11 + 2^-20 |lse|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SCALE = 192.0 ** -0.5


class Case:
    """A ragged batch: new rows and tokens per request; keys and values as views of one product,
    the rotary keys a view of 576-wide entries, `pad` unused rows and entries around everything."""

    def __init__(self, new, seqs, heads=3, e=1, seed=1, pad=0, scale=SCALE, q_mag=1.0):
        import torch
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.new, self.seqs, self.heads, self.e, self.scale = list(new), list(seqs), heads, e, scale
        self.entries = [-(-max(s, 0) // e) for s in self.seqs]
        cu = lambda v: [pad + sum(v[:i]) for i in range(len(v) + 1)]  # noqa: E731
        self.cu_q_l, self.cu_kv_l = cu(self.new), cu(self.entries)
        tq, tk = sum(self.new) + 2 * pad, max(1, sum(self.entries) + 2 * pad)
        self.q = r(tq, heads, 192) * q_mag
        kv = r(tk, heads, 256)
        self.kn, self.v = kv[..., :128], kv[..., 128:]
        self.kr = r(tk, 576)[:, 512:]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        self.cu_q, self.cu_kv, self.seq = i32(self.cu_q_l), i32(self.cu_kv_l), i32(self.seqs)

    def args(self):
        return self.q, self.kn, self.kr, self.v, self.cu_q, self.cu_kv, self.seq, self.scale

    def reference(self, b, h):
        import torch
        q0, k0, n, m = self.cu_q_l[b], self.cu_kv_l[b], self.new[b], self.entries[b]
        q = self.q[q0:q0 + n, h].double()
        k = torch.cat([self.kn[k0:k0 + m, h], self.kr[k0:k0 + m]], 1).double()
        v = self.v[k0:k0 + m, h].double()
        seen = torch.tensor([-(-max(self.seqs[b] - (n - 1 - i), 0) // self.e) for i in range(n)], device="cuda")
        s = (self.scale * (q @ k.T)).masked_fill(torch.arange(m, device="cuda") >= seen[:, None], -float("inf"))
        lse = torch.logsumexp(s, 1)
        w = torch.where(seen[:, None] > 0, torch.exp(s - torch.where(seen > 0, lse, 0)[:, None]), 0)
        return w @ v, lse, w @ v.abs(), seen

    def check(self, out, lse, requests=None, heads=None):
        import torch
        for b in range(len(self.new)) if requests is None else requests:
            if self.new[b] == 0:
                continue
            rows = slice(self.cu_q_l[b], self.cu_q_l[b] + self.new[b])
            for h in range(self.heads) if heads is None else heads:
                o, l, a, seen = self.reference(b, h)
                got, gl = out[rows, h].double(), lse[rows, h].double()
                none = seen == 0
                assert not got[none].any() and torch.isneginf(gl[none]).all(), f"request {b}: empty rows"
                err, tol = (got - o).abs(), (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * o.abs() + 1e-12
                assert not (err > tol).any(), \
                    f"request {b} head {h}: out off at {(err > tol).nonzero()[:3].tolist()}, {float((err / (a + 1e-9)).max())}"
                dl = (gl - l).abs()[~none]
                assert torch.all(dl <= 2.0 ** -11 + 2.0 ** -20 * l.abs()[~none]), f"request {b} head {h}: lse"


def run(lib, case, split=False, **kw):
    import torch
    ws = lib.new_mla_workspace(1) if split else torch.zeros(256, dtype=torch.uint8, device="cuda")
    out, lse = lib.dsa_mla_prefill(*case.args(), entry_tokens=case.e, workspace=ws, **kw)
    assert lib.get_error(ws) == 0
    return out, lse


@pytest.mark.parametrize("e", [1, 4])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 64, 100, 127, 128, 129, 130, 200, 255, 256, 257, 300, 384, 385, 400, 511, 512, 513, 767, 768,
                               769, 1000, 1025, 1300])
def test_prefill_one_prompt(gpu_lib, n, e):
    """Prompts of every kind of partial tile, an entry per token or per four."""
    case = Case([n], [n], heads=2, e=e, seed=n)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("n, seq, e", [(1, 1000, 1), (1, 1000, 4), (5, 257, 1), (5, 260, 4), (128, 1024, 1),
                                       (129, 2000, 4), (256, 1023, 1), (300, 4097, 4), (700, 5000, 3), (64, 9000, 64)])
def test_prefill_chunks(gpu_lib, n, seq, e):
    """New rows on top of earlier tokens."""
    case = Case([n], [seq], heads=3, e=e, seed=n + seq)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("n, seq, e, heads", [(1, 1024, 1, 1), (1, 30000, 4, 1), (3, 4097, 1, 2), (64, 9001, 1, 5),
                                              (130, 5000, 4, 3), (256, 20000, 4, 18), (257, 3000, 1, 1),
                                              (400, 8191, 1, 7), (512, 12000, 4, 20), (700, 6000, 1, 3),
                                              (1100, 1100, 1, 1), (5, 600, 1, 1), (20, 66000, 1, 3)])
def test_prefill_split(gpu_lib, n, seq, e, heads):
    """Few units over many entries: parts of each on clusters of their own, joined by the merge; and the
    same call unsplit.  One row, both kinds of unit, units of unlike length, parts that some rows (and one
    of two tiles) see nothing of."""
    case = Case([n], [seq], heads=heads, e=e, seed=n + heads)
    case.check(*run(gpu_lib, case, split=True))
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("new, seqs, e, heads", [([520], [9000], 1, 80), ([1024], [40000], 4, 64),
                                                 ([300, 40, 513], [7000, 5000, 6600], 1, 33)])
def test_prefill_split_last_round(gpu_lib, new, seqs, e, heads):
    """More units than clusters: the ones behind the last whole round in parts, the others whole."""
    case = Case(new, seqs, heads=heads, e=e, seed=heads)
    some = [0, 1, heads // 2, heads - 2, heads - 1]
    case.check(*run(gpu_lib, case, split=True), heads=some)
    case.check(*run(gpu_lib, case), heads=some)


@pytest.mark.parametrize("new, seqs, e, heads", [([1500, 700, 0, 2100, 600], [1500, 700, 5, 2100, 650], 1, 3),
                                                 ([1300, 900, 1100], [60000, 900, 4000], 4, 2),
                                                 ([2049, 1, 513, 2000], [2049, 3000, 513, 1500], 1, 7)])
def test_prefill_long_prompts(gpu_lib, new, seqs, e, heads):
    """Several prompts of more than a block of rows: their units ordered across requests, those of a chunk
    on a long past head by head."""
    case = Case(new, seqs, heads=heads, e=e, seed=sum(new))
    case.check(*run(gpu_lib, case))


def test_prefill_long_prompts_many(gpu_lib):
    """More groups of units than there are threads to order them."""
    case = Case([520 + b % 3 for b in range(200)], [520 + b % 7 for b in range(200)], heads=1, e=1, seed=41)
    case.check(*run(gpu_lib, case), requests=range(0, 200, 9))


def test_prefill_split_ragged(gpu_lib):
    """A long and a short request, one without rows and one shorter than its rows, in parts; the workspace
    reused by calls of other splits, the same bits again."""
    import torch
    case = Case([40, 0, 300, 9], [20000, 50, 310, 5], heads=3, e=1, seed=21)
    ws = gpu_lib.new_mla_workspace(1)
    f = lambda c: [t.clone() for t in gpu_lib.dsa_mla_prefill(*c.args(), entry_tokens=c.e, workspace=ws)]  # noqa: E731
    first = f(case)
    case.check(*first)
    other = Case([2], [70000], heads=1, e=4, seed=22)
    other.check(*f(other))
    again = f(case)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]) and gpu_lib.get_error(ws) == 0


@pytest.mark.parametrize("n, seq, e, heads", [(100, 30000, 4, 3), (300, 3001, 1, 2), (1, 9999, 1, 1)])
def test_prefill_split_beside_nan(gpu_lib, n, seq, e, heads):
    """Split, between rows and entries that belong to nobody: NaN there reaches nothing, and their
    outputs stay as they are."""
    import torch
    pad = 9
    case = Case([n], [seq], heads=heads, e=e, seed=n, pad=pad)
    m = case.entries[0]
    for t, rows in ((case.q, n), (case.kn, m), (case.v, m), (case.kr, m)):
        t[:pad] = float("nan")
        t[pad + rows:] = float("nan")
    out = torch.full((n + 2 * pad, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 2 * pad, heads), 7.0, device="cuda")
    case.check(*run(gpu_lib, case, split=True, out=out, lse=lse))
    for t in (out, lse):
        assert torch.all(t[:pad] == 7.0) and torch.all(t[pad + n:] == 7.0)


def test_prefill_and_decode_share_a_workspace(gpu_lib):
    """One after another on one stream, captured and replayed: the same bits as on workspaces of their own."""
    import torch
    case = Case([50], [30000], heads=4, e=4, seed=31)
    g = torch.Generator().manual_seed(32)
    q = torch.randn(2, 64, 576, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(40, 64, 576, generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(64, dtype=torch.int32).remainder(40).view(2, 32).cuda()
    seq = torch.tensor([8000, 3000], dtype=torch.int32).cuda()
    ws = [gpu_lib.new_mla_workspace(2) for _ in range(3)]

    def both(a, b):
        o = gpu_lib.dsa_mla_prefill(*case.args(), entry_tokens=4, workspace=a)
        d = gpu_lib.dsa_mla_decode(q, kv, table, seq, 8192, SCALE, workspace=b)
        return [*o, *d, *gpu_lib.dsa_mla_prefill(*case.args(), entry_tokens=4, workspace=a)]

    want = both(ws[0], ws[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(ws[2], ws[2])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(gpu_lib.get_error(w) == 0 for w in ws)


def test_prefill_split_graph_lengths(gpu_lib):
    """Captured on one batch, replayed on lengths that are split otherwise, or not at all."""
    import torch
    case = Case([6, 50], [30000, 2000], heads=2, e=1, seed=23)
    ws = gpu_lib.new_mla_workspace(1)
    out = torch.empty(56, 2, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(56, 2, device="cuda")
    args = case.args()
    gpu_lib.dsa_mla_prefill(*args, entry_tokens=1, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.dsa_mla_prefill(*args, entry_tokens=1, out=out, lse=lse, workspace=ws)
    for seqs in ([30000, 2000], [100, 60], [6, 1999], [29000, 50]):
        case.seqs = seqs
        case.seq.copy_(torch.tensor(seqs, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        case.check(out, lse)
    assert gpu_lib.get_error(ws) == 0


@pytest.mark.parametrize("heads", [1, 2, 5, 64, 128])
def test_prefill_heads(gpu_lib, heads):
    case = Case([70, 300], [70, 350], heads=heads, e=4, seed=heads)
    case.check(*run(gpu_lib, case))


@pytest.mark.parametrize("e", [1, 4])
def test_prefill_ragged(gpu_lib, e):
    """Many requests, some without rows, some without tokens, shorter than their rows (rows that see
    nothing), behind unused rows and entries that hold NaN; rows outside the batch stay as they were."""
    import torch
    new = [1, 0, 300, 7, 128, 0, 513, 64, 2, 256, 255, 33, 10]
    seqs = [1, 50, 300, 2000, 128, 0, 700, 64, 0, 256, 400, 20, 7]
    case = Case(new, seqs, heads=2, e=e, seed=3, pad=37)
    lo, hi = case.cu_q_l[0], case.cu_q_l[-1]
    case.q[:lo] = float("nan")
    case.q[hi:] = float("nan")
    for t in (case.kn, case.v, case.kr):
        t[:case.cu_kv_l[0]] = float("nan")
        t[case.cu_kv_l[-1]:] = float("nan")
    out = torch.full((case.q.shape[0], 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.q.shape[0], 2), 7.0, device="cuda")
    run(gpu_lib, case, out=out, lse=lse)
    case.check(out, lse)
    for t in (out, lse):
        assert torch.all(t[:lo] == 7.0) and torch.all(t[hi:] == 7.0)


def test_prefill_requests_do_not_touch_each_other(gpu_lib):
    """Each request alone gives the bits it has in the batch, and a NaN request spoils only itself."""
    import torch
    case = Case([200, 129, 300], [200, 400, 301], heads=2, seed=4)
    out, lse = run(gpu_lib, case)
    for t in (case.q[200:329], case.v[200:600], case.kn[200:600]):
        t.fill_(float("nan"))
    case.kr[200:600] = float("inf")
    got, gl = run(gpu_lib, case)
    for rows in (slice(0, 200), slice(329, 629)):
        assert torch.equal(out[rows], got[rows]) and torch.equal(lse[rows], gl[rows])
    one = Case([200], [200], heads=2, seed=4)
    one.q, one.kn, one.kr, one.v = case.q[:200], case.kn[:200], case.kr[:200], case.v[:200]
    o1, l1 = run(gpu_lib, one)
    assert torch.equal(o1, out[:200]) and torch.equal(l1, lse[:200])


def test_prefill_more_entries_than_tokens(gpu_lib):
    """Entries of a request past its live length (a padded batch) are never used."""
    import torch
    case = Case([100, 50], [300, 260], heads=2, e=4, seed=5)
    want = run(gpu_lib, case)
    case.seq -= torch.tensor([40, 0], dtype=torch.int32, device="cuda")
    case.seqs = [260, 260]
    live = 65
    for t in (case.kn, case.v, case.kr):
        t[live:75] = float("nan")
    out, lse = run(gpu_lib, case)
    assert torch.isfinite(out.float()).all()
    assert torch.equal(out[100:], want[0][100:])
    case.entries[0] = live
    case.check(out, lse, requests=[0])


def test_prefill_running_max(gpu_lib):
    """Keys that grow along the prompt: the maximum rises by more than 2^8 from tile to tile and the
    accumulator is rescaled (late tiles dominate)."""
    case = Case([600], [1400], heads=2, seed=6, scale=0.125)
    for i in range(11):
        case.kn[128 * i:128 * (i + 1)] *= 2.0 ** (i / 2.5 - 2)
    out, lse = run(gpu_lib, case)
    case.check(out, lse)


def test_prefill_zero_scale_is_the_mean(gpu_lib):
    import torch
    case = Case([300], [300], heads=1, seed=7, scale=0.0)
    out, lse = run(gpu_lib, case)
    case.check(out, lse)
    assert torch.allclose(lse[:, 0].cpu(), torch.arange(1, 301).float().log(), atol=1e-5)


@pytest.mark.parametrize("e", [1, 4])
def test_prefill_matches_the_absorbed_decode(gpu_lib, e):
    """The two forms on one latent cache: keys and values expanded by per-head matrices (exact in
    bf16: each picks latent dims), the last row against the decode over the same entries."""
    import torch
    heads, n = 64, 4 * 700 if e == 4 else 700
    g = torch.Generator().manual_seed(8)
    entries = 700
    pages = -(-entries // 64)
    lat = torch.zeros(pages * 64, 576, dtype=torch.bfloat16)
    lat[:entries] = torch.randn(entries, 576, generator=g).to(torch.bfloat16)
    lat = lat.cuda()
    kdim, vdim = (torch.stack([torch.randperm(512, generator=g)[:128] for _ in range(heads)]).cuda() for _ in "kv")
    kn = torch.stack([lat[:entries, kdim[h]] for h in range(heads)], 1).contiguous()
    v = torch.stack([lat[:entries, vdim[h]] for h in range(heads)], 1).contiguous()
    rows = 150
    q = torch.randn(rows, heads, 192, generator=g).to(torch.bfloat16).cuda()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = gpu_lib.dsa_mla_prefill(q, kn, lat[:entries, 512:], v, i32(0, rows), i32(0, entries), i32(n), SCALE,
                                       entry_tokens=e)
    qa = torch.zeros(1, heads, 576, dtype=torch.bfloat16, device="cuda")
    for h in range(heads):
        qa[0, h, kdim[h]] = q[-1, h, :128]
    qa[..., 512:] = q[-1, :, 128:]
    ctx = -(-entries * 4 // 256) * 256
    dec, dl = gpu_lib.dsa_mla_decode(qa, lat.view(pages, 64, 576), torch.arange(pages, dtype=torch.int32,
                                                                               device="cuda")[None], i32(entries * 4),
                                     ctx, SCALE)
    want = torch.stack([dec[0, h, vdim[h]] for h in range(heads)])
    assert (out[-1].float() - want.float()).abs().max() < 2.0 ** -5
    assert (lse[-1] - dl[0]).abs().max() < 2.0 ** -10


def test_prefill_layouts(gpu_lib):
    """Heads before rows, and tensors of their own: the same bits as the views."""
    import torch
    case = Case([150, 90], [150, 200], heads=4, seed=9)
    want = run(gpu_lib, case)
    turned = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    got = gpu_lib.dsa_mla_prefill(turned(case.q), turned(case.kn), case.kr.contiguous(), case.v.contiguous(),
                                  case.cu_q, case.cu_kv, case.seq, case.scale, entry_tokens=1)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_prefill_bad_ranges(gpu_lib):
    """Rows or entries out of order or range, too few entries, a negative length: flagged, never
    dereferenced, and the other requests are right."""
    import torch
    case = Case([100, 60, 200, 40], [100, 60, 250, 40], heads=2, seed=10)
    good = run(gpu_lib, case)

    def call(cu_q=None, cu_kv=None, seq=None):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        i32 = lambda v, d: d if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        out = torch.zeros_like(good[0])
        gpu_lib.dsa_mla_prefill(case.q, case.kn, case.kr, case.v, i32(cu_q, case.cu_q), i32(cu_kv, case.cu_kv),
                                i32(seq, case.seq), case.scale, entry_tokens=1, out=out, workspace=ws)
        return out, gpu_lib.get_error(ws)

    rows = lambda b: slice(case.cu_q_l[b], case.cu_q_l[b + 1])  # noqa: E731
    out, err = call(cu_q=case.cu_q_l[:4] + [1 << 30])
    assert err == gpu_lib.DEVERR_BAD_RANGE
    assert all(torch.equal(out[rows(b)], good[0][rows(b)]) for b in range(3)) and not out[rows(3)].any()
    out, err = call(cu_kv=case.cu_kv_l[:4] + [case.v.shape[0] + 1])
    assert err == gpu_lib.DEVERR_BAD_RANGE and torch.equal(out[rows(1)], good[0][rows(1)])
    out, err = call(cu_kv=[-4] + case.cu_kv_l[1:])
    assert err == gpu_lib.DEVERR_BAD_RANGE and not out[rows(0)].any()
    out, err = call(seq=[100, 60, 251, 40])     # one entry more than there are
    assert err == gpu_lib.DEVERR_BAD_RANGE and torch.equal(out[rows(3)], good[0][rows(3)])
    out, err = call(seq=[100, -60, 250, 40])
    assert err == gpu_lib.DEVERR_SEQ_LEN_CLAMPED and not out[rows(1)].any()
    assert torch.equal(out[rows(2)], good[0][rows(2)])


@pytest.mark.parametrize("new, seqs", [([60, 40, 30], [9000, 5000, 7000]), ([700, 900, 1200], [700, 900, 1200])])
def test_prefill_bad_ranges_split_and_ordered(gpu_lib, new, seqs):
    """The same where rows are split along their entries, and where units are ordered across requests."""
    import torch
    case = Case(new, seqs, heads=2, seed=15)
    run(gpu_lib, case, split=True)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = gpu_lib.new_mla_workspace(1)
    cu_q, cu_kv = case.cu_q_l, case.cu_kv_l
    for bad_q, bad_kv, bad_seq, wrong in ((cu_q[:3] + [1 << 30], cu_kv, seqs, 2), ([-5] + cu_q[1:], cu_kv, seqs, 0),
                                          (cu_q, cu_kv[:3] + [case.v.shape[0] + 1], seqs, 2),
                                          (cu_q, cu_kv, [seqs[0] + 1] + seqs[1:], 0), (cu_q, cu_kv, [-3] + seqs[1:], 0)):
        out = torch.full((sum(new), 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((sum(new), 2), 7.0, device="cuda")
        gpu_lib.dsa_mla_prefill(case.q, case.kn, case.kr, case.v, i32(bad_q), i32(bad_kv), i32(bad_seq), case.scale,
                                entry_tokens=1, out=out, lse=lse, workspace=ws)
        want = gpu_lib.DEVERR_SEQ_LEN_CLAMPED if bad_seq[0] < 0 else gpu_lib.DEVERR_BAD_RANGE
        assert gpu_lib.get_error(ws) == want
        case.check(out, lse, requests=[b for b in range(3) if b != wrong])


def test_prefill_split_two_streams(gpu_lib):
    """Two split calls, a decode and a norm at once on their own streams and workspaces: the same bits as alone."""
    import torch
    a, b = Case([9], [40000], heads=2, e=1, seed=16), Case([300], [20000], heads=3, e=4, seed=17)
    g = torch.Generator().manual_seed(18)
    q, kv = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((4, 64, 576), (64, 64, 576)))
    table = torch.arange(128, dtype=torch.int32).remainder(64).view(4, 32).cuda()
    seq = torch.tensor([8000, 100, 3000, 0], dtype=torch.int32).cuda()
    x = torch.randn(3000, 512, generator=g).to(torch.bfloat16).cuda()
    calls = [lambda ws: gpu_lib.dsa_mla_prefill(*a.args(), entry_tokens=1, workspace=ws),
             lambda ws: gpu_lib.dsa_mla_prefill(*b.args(), entry_tokens=4, workspace=ws),
             lambda ws: gpu_lib.dsa_mla_decode(q, kv, table, seq, 8192, SCALE, workspace=ws),
             lambda ws: gpu_lib.dsa_rmsnorm_fp8(x, x[0].contiguous(), 1e-6, 128)[:2]]
    spaces = [gpu_lib.new_mla_workspace(4) for _ in calls]
    want = [[t.clone() for t in f(ws)] for f, ws in zip(calls, spaces)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        got = []
        for f, ws, s in zip(calls, spaces, streams):
            with torch.cuda.stream(s):
                got.append(f(ws))
        torch.cuda.synchronize()
        for p, r in zip(want, got):
            assert all(torch.equal(m.view(torch.uint8), n.view(torch.uint8)) for m, n in zip(p, r))
    assert all(gpu_lib.get_error(ws) == 0 for ws in spaces)


def test_prefill_no_entries(gpu_lib):
    """No entry at all, and no row at all."""
    import torch
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = gpu_lib.dsa_mla_prefill(z(5, 2, 192) + 1, z(0, 2, 128), z(0, 64), z(0, 2, 128), i32(0, 5), i32(0, 0),
                                       i32(0), SCALE)
    assert not out.any() and torch.isneginf(lse).all()
    out, lse = gpu_lib.dsa_mla_prefill(z(0, 2, 192), z(9, 2, 128), z(9, 64), z(9, 2, 128), i32(0, 0), i32(0, 9),
                                       i32(9), SCALE)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)


@pytest.mark.slow
def test_prefill_long(gpu_lib):
    """A 4,100-token prompt, and a chunk over 20,000 entries."""
    case = Case([4100], [4100], heads=2, e=1, seed=11, q_mag=2.0)
    case.check(*run(gpu_lib, case))
    case = Case([500, 3], [80000, 60001], heads=2, e=4, seed=12, q_mag=2.0)
    case.check(*run(gpu_lib, case))


def test_prefill_graph_streams_determinism(gpu_lib):
    """Captured, replayed with other lengths; two calls at once on two streams; the same bits twice."""
    import torch
    case = Case([100, 200, 84], [100, 300, 84], heads=2, seed=13)
    want = run(gpu_lib, case)
    again = run(gpu_lib, case)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    cu_q = torch.zeros_like(case.cu_q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.dsa_mla_prefill(case.q, case.kn, case.kr, case.v, cu_q, case.cu_kv, case.seq, case.scale,
                                entry_tokens=1, out=out, lse=lse, workspace=ws)
    cu_q.copy_(case.cu_q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and gpu_lib.get_error(ws) == 0
    other = Case([50], [2000], heads=5, e=4, seed=14)
    want2 = run(gpu_lib, other)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a = gpu_lib.dsa_mla_prefill(*case.args(), entry_tokens=1)
        with torch.cuda.stream(s2):
            b = gpu_lib.dsa_mla_prefill(*other.args(), entry_tokens=4)
    torch.cuda.synchronize()
    assert torch.equal(a[0], want[0]) and torch.equal(b[0], want2[0])


def test_prefill_refusals(gpu_lib):
    import torch
    c = Case([10], [10], heads=2)
    q, kn, kr, v, cq, ck, s, scale = c.args()
    f = gpu_lib.dsa_mla_prefill
    with pytest.raises(ValueError):
        f(q[..., :128], kn, kr, v, cq, ck, s, scale)
    with pytest.raises(ValueError):
        f(q, kn[:5], kr, v, cq, ck, s, scale)
    with pytest.raises(TypeError):
        f(q.float(), kn, kr, v, cq, ck, s, scale)
    with pytest.raises(ValueError):
        f(q, kn, kr, v, cq[:1], ck, s, scale)
    with pytest.raises(ValueError):
        f(q, kn, kr.t().contiguous().t(), v, cq, ck, s, scale)
    with pytest.raises(gpu_lib.DsaError):
        f(q, kn, kr, v, cq, ck, s, -1.0)
    with pytest.raises(gpu_lib.DsaError):
        f(q, kn, kr, v, cq, ck, s, scale, entry_tokens=0)
    odd = torch.zeros(10, 65, dtype=torch.bfloat16, device="cuda")[:, :64]   # rows not on 16-byte steps
    with pytest.raises(gpu_lib.DsaError):
        f(q, kn, odd, v, cq, ck, s, scale)
    with pytest.raises(gpu_lib.DsaError):
        f(q, kn, kr, v.new_zeros(1, 2, 128).expand(10, 2, 128), cq, ck, s, scale)   # stride 0
