"""GPU tests of the norms and the latent attentions as a decoder layer runs them: one after another
on their own outputs, beside the indexer and its sparse attention, on one cache and in one graph.

Every step is held to fp64 of the inputs it was given (the step before's own outputs), by the
bounds of that operator's own tests: norms 2^-8 + 2^-17 relatively; index scores 3e-3 of the row's
largest; dense attention (2^-8 + 2^-10) o_abs + 2^-8 |o| and lse 2^-11 + 2^-20 |lse|; sparse
attention 2^-7 o_abs + 1e-6 and lse 2^-8 + 1e-5 |lse|.  o_abs = sum_t w_t |v_t|."""
import pytest

pytestmark = pytest.mark.gpu

EPS, SCALE, D = 1e-6, 192.0 ** -0.5, 512


def bf16(g, *shape, mul=1.0):
    import torch
    return (torch.randn(*shape, generator=g) * mul).to(torch.bfloat16).cuda()


def paged(seqs, max_context, g):
    """A table of live pages in scattered order, and the number of pages."""
    import torch
    pages = [-(-s // 256) for s in seqs]
    perm = torch.randperm(sum(pages) + 2, generator=g).to(torch.int32)
    table = torch.full((len(seqs), max_context // 256), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = perm[sum(pages[:b]):sum(pages[:b]) + n]
    return table.cuda(), sum(pages) + 2


def entries(cache, table, b, n):
    import torch
    t = torch.arange(n, device="cuda")
    return cache[table[b].long()[t // 64], t % 64].double()


def norm64(h, weight):
    import torch
    h = h.double()
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * weight.double()


def near(got, want, tol, what):
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"


def check_attention(o, lse, q, kv, what, sparse=False):
    """o [heads, dv], lse [heads] of q [heads, 576] over kv [n, 576]."""
    import torch
    s = SCALE * (q.double() @ kv.T)
    w = torch.softmax(s, 1)
    ref, a, l = w @ kv[:, :512], w @ kv[:, :512].abs(), torch.logsumexp(s, 1)
    if sparse:
        near(o, ref, 2.0 ** -7 * a + 1e-6, what)
        near(lse, l, 2.0 ** -8 + 1e-5 * l.abs(), what + " lse")
    else:
        near(o, ref, (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * ref.abs() + 1e-12, what)
        near(lse, l, 2.0 ** -11 + 2.0 ** -20 * l.abs(), what + " lse")


class Layer:
    """One decode step: residual + norm, projection of the hidden rows, index keys' scores and top-k,
    then attention over the listed entries and over all of them."""

    def __init__(self, lib, seqs, max_context, k, seed):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.lib, self.B, self.max_context, self.k = lib, len(seqs), max_context, k
        self.table, pages = paged([max_context] * self.B, max_context, g)
        self.seq = torch.tensor(seqs, dtype=torch.int32).cuda()
        self.x, self.r = bf16(g, self.B, D), bf16(g, self.B, D, mul=3.0)
        self.weight = torch.randn(D, generator=g).cuda()
        self.w_q, self.w_w = bf16(g, 2048, D, mul=D ** -0.5), bf16(g, 32, D, mul=D ** -0.5)
        self.keys, self.kv = bf16(g, pages, 64, 64), bf16(g, pages, 64, 576)
        self.q_mla = bf16(g, self.B, 64, 576)
        e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        f32, B = torch.float32, self.B
        self.h, self.sum = e(B, D), e(B, D)
        self.q, self.w = e(B, 32, 64), e(B, 32, t=f32)
        self.topk = e(B, k, t=torch.int32)
        self.so, self.sl = e(B, 64, 512, t=f32), e(B, 64, t=f32)
        self.do, self.dl = e(B, 64, 512), e(B, 64, t=f32)
        z = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws = [lib.new_workspace(B, max_context, k), z(lib.qw_proj_workspace_size(B, D)),
                   z(lib.sparse_mla_workspace_size(B, k)), lib.new_mla_workspace(B)]

    def step(self):
        b = self.lib
        b.dsa_rmsnorm(self.x, self.weight, EPS, residual=self.r, out=self.h, residual_out=self.sum)
        b.dsa_indexer_qw_proj(self.h, self.w_q, self.w_w, q_out=self.q, w_out=self.w, workspace=self.ws[1])
        b.dsa_indexer_fused(self.q, self.w, self.keys, self.table, self.seq, self.max_context, self.k,
                            topk_idx=self.topk, workspace=self.ws[0])
        b.dsa_sparse_mla_decode(self.q_mla, self.kv, self.table, self.seq, self.max_context, self.topk, SCALE,
                                out=self.so, lse=self.sl, workspace=self.ws[2])
        b.dsa_mla_decode(self.q_mla, self.kv, self.table, self.seq, self.max_context, SCALE, out=self.do,
                         lse=self.dl, workspace=self.ws[3])

    def outputs(self):
        return [t.clone() for t in (self.h, self.sum, self.q, self.w, self.topk, self.so, self.sl, self.do, self.dl)]

    def check(self):
        import torch
        assert all(self.lib.get_error(ws) == 0 for ws in self.ws)
        h = self.x.double() + self.r.double()
        near(self.sum, h, (2.0 ** -8 + 2.0 ** -17) * h.abs(), "sum")
        y = norm64(h, self.weight)
        near(self.h, y, (2.0 ** -8 + 2.0 ** -17) * y.abs() + 1e-38, "norm")
        for b in range(self.B):
            n = -(-int(self.seq[b]) // 4)
            got = self.topk[b]
            got = got[got >= 0].long()
            assert got.numel() == min(n, self.k) and (got[1:] > got[:-1]).all() and (got < n).all()
            if n == 0:
                assert not self.do[b].any() and not self.so[b].any() and torch.isneginf(self.dl[b]).all()
                continue
            s = self.w[b].double() @ torch.relu(self.q[b].double() @ entries(self.keys, self.table, b, n).T)
            left = torch.ones(n, dtype=torch.bool, device="cuda")
            left[got] = False
            if left.any():  # nothing left out is ahead of what was taken by more than the scores' error
                assert s[left].max() - s[got].min() <= 2 * 3e-3 * s.abs().max()
            kv = entries(self.kv, self.table, b, n)
            check_attention(self.do[b], self.dl[b], self.q_mla[b], kv, f"dense {b}")
            check_attention(self.so[b], self.sl[b], self.q_mla[b], kv[got], f"sparse {b}", sparse=True)


@pytest.mark.parametrize("k", [64, 2048])
def test_decode_layer(gpu_lib, k):
    """Eager, and captured on another stream and replayed on other rows and lengths; where top-k lists
    every live entry (2048 of at most 2048), both attentions are of the same entries."""
    import torch
    layer = Layer(gpu_lib, [8192, 1, 0, 517, 2600], 8192, k, seed=31 + k)
    layer.step()
    torch.cuda.synchronize()
    layer.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        layer.step()
    layer.seq.copy_(torch.tensor([3, 8000, 4097, 0, 256], dtype=torch.int32))
    layer.x.copy_(layer.x.flip(0) * 2)
    graph.replay()
    torch.cuda.synchronize()
    layer.check()
    replayed = layer.outputs()
    layer.step()
    torch.cuda.synchronize()
    for a, b in zip(replayed, layer.outputs()):
        assert torch.equal(a, b)


def test_fp8_keys_from_the_norm(gpu_lib):
    """Index keys normed straight into the fp8 cache's pages (64 codes and a scale each), and scored."""
    import torch
    g = torch.Generator().manual_seed(41)
    seqs, max_context = [4096, 300, 1999], 4096
    table, pages = paged(seqs, max_context, g)
    raw, weight = bf16(g, pages * 64, 128, mul=2.0), torch.randn(64, generator=g).cuda()
    codes = torch.empty(pages, 64, 64, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(pages, 64, device="cuda")
    gpu_lib.dsa_rmsnorm_fp8(raw[:, 64:], weight, EPS, 64, codes=codes.view(-1, 64), scales=scales.view(-1, 1))
    keys = codes.cpu().view(torch.float8_e4m3fn).double().cuda() * scales.double()[..., None]
    y = norm64(raw[:, 64:], weight).view_as(keys)
    amax = y.abs().amax(-1, keepdim=True)
    near(keys, y, torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 / 448 * amax) + 2.0 ** -16 * amax, "keys")
    q, w = bf16(g, 3, 32, 64), (torch.randn(3, 32, generator=g) / 32).cuda()
    seq = torch.tensor(seqs, dtype=torch.int32).cuda()
    ws = gpu_lib.new_workspace(3, max_context, 16)
    scores = gpu_lib.dsa_indexer_scores_fp8(q, w, codes, scales, table, seq, max_context, workspace=ws)
    assert gpu_lib.get_error(ws) == 0
    for b, s in enumerate(seqs):
        n = -(-s // 4)
        want = w[b].double() @ torch.relu(q[b].double() @ entries(keys, table, b, n).T)
        near(scores[b, :n], want, 3e-3 * want.abs().max(), f"scores {b}")
        assert torch.isneginf(scores[b, n:]).all()


@pytest.mark.parametrize("new, seqs", [([40, 4, 300], [40, 3001, 900]), ([4, 700, 5], [4, 700, 1023])])
def test_prefill_and_decode_on_one_cache(gpu_lib, new, seqs):
    """A chunk's last four rows by the expanded form, and by the absorbed one with four query tokens.

    Latents are normed rows of a wider product.  The up-projections pick 128 of the 512 latent dims
    (other ones for keys and values, by head), so that both forms have the same exact operands: what
    they leave is each one's own error."""
    import torch
    g = torch.Generator().manual_seed(sum(seqs))
    heads, B, max_context = 64, len(seqs), 4096
    count = [-(-s // 4) for s in seqs]
    cu = lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=torch.int32).cuda()  # noqa: E731
    raw, weight = bf16(g, sum(count), 640, mul=2.0), bf16(g, 512)
    latent, _ = gpu_lib.dsa_rmsnorm(raw[:, :512], weight, EPS)
    near(latent, norm64(raw[:, :512], weight), (2.0 ** -8 + 2.0 ** -17) * norm64(raw[:, :512], weight).abs() + 1e-38,
         "latent")
    rows = torch.cat([latent, raw[:, 512:576]], 1)  # 576-wide entries
    q = bf16(g, sum(new), heads, 192)
    part = torch.arange(heads, device="cuda") % 4
    slices = latent.view(-1, 4, 128)
    k_nope, v = slices[:, part].contiguous(), slices[:, (part + 1) % 4].contiguous()
    ws = gpu_lib.new_mla_workspace(B, 4)
    out, lse = gpu_lib.dsa_mla_prefill(q, k_nope, rows[:, 512:], v, cu(new), cu(count),
                                       torch.tensor(seqs, dtype=torch.int32).cuda(), SCALE, entry_tokens=4,
                                       workspace=ws)
    # the same entries in pages, and the same queries absorbed
    table, pages = paged(seqs, max_context, g)
    cache = torch.full((pages, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    last = torch.empty(B, 4, heads, 192, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        t = torch.arange(count[b], device="cuda")
        cache[table[b].long()[t // 64], t % 64] = rows[sum(count[:b]):sum(count[:b + 1])]
        last[b] = q[sum(new[:b + 1]) - 4:sum(new[:b + 1])]
    absorbed = torch.zeros(B, 4, heads, 4, 128, dtype=torch.bfloat16, device="cuda")
    absorbed[:, :, torch.arange(heads), part] = last[..., :128]
    absorbed = torch.cat([absorbed.view(B, 4, heads, 512), last[..., 128:]], -1)
    seq = torch.tensor(seqs, dtype=torch.int32).cuda()
    o4, l4 = gpu_lib.dsa_mla_decode(absorbed, cache, table, seq, max_context, SCALE, workspace=ws)
    assert gpu_lib.get_error(ws) == 0
    for b in range(B):
        for j in range(4):
            n = -(-max(seqs[b] - (3 - j), 0) // 4)
            kv = entries(cache, table, b, n)
            check_attention(o4[b, j], l4[b, j], absorbed[b, j], kv, f"decode {b} {j}")
            i = sum(new[:b + 1]) - 4 + j
            s = SCALE * (absorbed[b, j].double() @ kv.T)
            w = torch.softmax(s, 1)
            values = kv[:, :512].view(n, 4, 128)[:, (part + 1) % 4]  # [n, heads, 128]
            ref, a = torch.einsum("ht,thd->hd", w, values), torch.einsum("ht,thd->hd", w, values.abs())
            near(out[i], ref, (2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * ref.abs() + 1e-12, f"prefill {b} {j}")
            l = torch.logsumexp(s, 1)
            near(lse[i], l, 2.0 ** -11 + 2.0 ** -20 * l.abs(), f"prefill {b} {j} lse")
