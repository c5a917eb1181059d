"""GPU test of the paged caches' operators as a serving loop runs them: pages and slots for the next step, the new
entries normed, rotated, quantised and written at their slots, and a tree of drafted tokens verified over the
cache; requests arrive, grow, roll back and end, with one set of caches and one workspace, eager and replayed.
Each step is held to fp64 of what it was given, by the bounds of that operator's own tests."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

EPS, SCALE, B, T, MAX, PAGES, ROOM = 1e-6, 192.0 ** -0.5, 6, 7, 8192, 120, 4096


class Server:
    """The device's state, and what a plain host program knows of it."""

    def __init__(self, lib, seed):
        import torch
        self.lib, self.g, self.rng = lib, torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.want, self.table = i32(B), i32(B), torch.full((B, MAX // 256), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(PAGES, generator=self.g).to(torch.int32).cuda()
        self.count = torch.full((1,), PAGES, dtype=torch.int32, device="cuda")
        self.cu, self.slots = i32(B + 1), torch.zeros(ROOM, dtype=torch.int64, device="cuda")
        self.positions = i32(ROOM)
        self.kv = torch.zeros(PAGES, 64, 576, dtype=torch.bfloat16, device="cuda")
        self.codes = torch.zeros(PAGES, 64, 64, dtype=torch.uint8, device="cuda")
        self.scales = torch.ones(PAGES, 64, device="cuda")
        self.rows = torch.zeros(ROOM, 576 + 64, dtype=torch.bfloat16, device="cuda")
        self.weight, self.key_weight = (1 + 0.2 * self.rand(512)), (1 + 0.2 * self.rand(64))
        angle = torch.rand(MAX // 4, 32, generator=self.g).double() * 6
        self.table_cs = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.q = torch.zeros(B, T, 64, 576, dtype=torch.bfloat16, device="cuda")
        self.draft = torch.zeros(B, T, 576, dtype=torch.bfloat16, device="cuda")
        self.mask, self.counts = torch.zeros(B, T, dtype=torch.int64, device="cuda"), i32(B)
        self.out = torch.zeros(B, T, 64, 512, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(B, T, 64, device="cuda")
        self.ws = lib.new_tree_workspace(B, T)
        self.entries = [[] for _ in range(B)]      # per request: its entries' rows as they should be, in fp64

    def rand(self, *shape):
        import torch
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16).cuda()

    def step(self):
        """What the GPU does in a step, on the state's own buffers."""
        self.lib.dsa_pages_update(self.lens, self.want, MAX, self.table, self.free, self.count, ROOM,
                                  seq_lens_out=self.lens, free_count_out=self.count, cu_slots=self.cu, slots=self.slots,
                                  positions=self.positions, workspace=self.ws)
        self.lib.dsa_cache_append(self.slots, latent=self.rows[:, :576], latent_weight=self.weight, cos_sin=self.table_cs,
                                  positions=self.positions, kv_cache=self.kv, index_keys=self.rows[:, 576:],
                                  index_weight=self.key_weight, key_codes=self.codes, key_scales=self.scales, eps=EPS,
                                  workspace=self.ws)
        self.lib.dsa_mla_tree_decode(self.q, self.kv, self.table, self.lens, MAX, self.draft, self.mask, SCALE,
                                     token_counts=self.counts, out=self.out, lse=self.lse, workspace=self.ws)

    def new_inputs(self, want):
        import torch
        self.want.copy_(torch.tensor(want, dtype=torch.int32))
        self.rows.copy_(self.rand(ROOM, 640))
        self.q.copy_(self.rand(B, T, 64, 576))
        self.draft.copy_(self.rand(B, T, 576))
        counts = self.rng.integers(0, T + 1, B)
        seen = np.zeros((B, T), dtype=np.int64)
        for b in range(B):
            for j in range(T):
                parent = self.rng.integers(-1, j) if j else -1
                seen[b, j] = (seen[b, parent] if parent >= 0 else 0) | 1 << j
        self.mask.copy_(torch.from_numpy(seen))
        self.counts.copy_(torch.from_numpy(counts.astype(np.int32)))

    def check(self, before, want):
        import torch
        lens, cu, slots = self.lens.tolist(), self.cu.tolist(), self.slots.tolist()
        assert lens == want and self.lib.get_error(self.ws) == 0
        table = self.table.tolist()
        live = [p for b in range(B) for p in table[b][:-(-lens[b] // 256)]]
        free = self.free[: int(self.count)].tolist()
        assert sorted(live + free) == list(range(PAGES))                       # every page is somewhere, once
        x = self.rows.double()
        c, s = self.table_cs.double()[self.positions.clamp(min=0).long()].chunk(2, 1)
        a, d = x[:, 512:576:2], x[:, 513:576:2]
        normed = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w.double()  # noqa: E731
        rotated = torch.stack([a * c - d * s, a * s + d * c], 2).flatten(1)
        made = torch.cat([normed(x[:, :512], self.weight), rotated], 1)
        size = torch.cat([made[:, :512].abs(), torch.stack([(a * c).abs() + (d * s).abs(), (a * s).abs() + (d * c).abs()],
                                                          2).flatten(1)], 1)
        key = normed(x[:, 576:], self.key_weight)
        flat = self.kv.view(-1, 576)
        for b in range(B):
            n, w = before[b], want[b]
            self.entries[b] = self.entries[b][: -(-min(n, w) // 4)]
            if w > n:
                self.entries[b] = self.entries[b][: n // 4]
                assert cu[b + 1] - cu[b] == -(-w // 4) - n // 4
                self.entries[b] += [(made[i], size[i], key[i]) for i in range(cu[b], cu[b + 1])]
            if not lens[b]:
                continue
            t = torch.arange(-(-lens[b] // 4), device="cuda")
            at = self.table[b].long()[t // 64] * 64 + t % 64
            if w > n:
                assert slots[cu[b]:cu[b + 1]] == at[n // 4:].tolist()
            got = flat[at].double()
            ref = torch.stack([e[0] for e in self.entries[b]])
            bound = torch.stack([e[1] for e in self.entries[b]])
            assert not ((got - ref).abs() > (2.0 ** -8 + 2.0 ** -18) * ref.abs() + 2.0 ** -22 * bound).any(), b
            k = torch.stack([e[2] for e in self.entries[b]])
            codes = self.codes.view(-1, 64)[at].view(torch.float8_e4m3fn).float().double()
            sc = self.scales.view(-1)[at].double()[:, None]
            top = k.abs().amax(1, keepdim=True)
            assert not ((codes * sc - k).abs() > 2.0 ** -4 * k.abs() + 2.0 ** -10 * sc + 2.0 ** -17 * top).any(), b
        for b in range(B):
            t = torch.arange(-(-lens[b] // 4), device="cuda")
            cache = flat[self.table[b].long()[t // 64] * 64 + t % 64]
            for j in range(int(self.counts[b])):
                own = [i for i in range(T) if int(self.mask[b, j]) >> i & 1]
                kv = torch.cat([cache, self.draft[b, own]]).double()
                sc = SCALE * (self.q[b, j].double() @ kv.T)
                w = torch.softmax(sc, 1)
                o, ab, l = w @ kv[:, :512], w @ kv[:, :512].abs(), torch.logsumexp(sc, 1)
                err = (self.out[b, j].double() - o).abs()
                assert not (err > (2.0 ** -8 + 2.0 ** -10) * ab + 2.0 ** -8 * o.abs() + 1e-12).any(), (b, j)
                assert torch.all((self.lse[b, j].double() - l).abs() <= 2.0 ** -11 + 2.0 ** -20 * l.abs()), (b, j)


@pytest.mark.parametrize("replayed", [False, True])
def test_serving_steps(gpu_lib, replayed):
    import torch
    server = Server(gpu_lib, 3 + replayed)
    graph = None
    if replayed:
        server.step()                             # nothing wanted, nothing done
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            server.step()
    now = [0] * B
    for step in range(7):
        want = []
        for n in now:
            r = server.rng.random()
            if n == 0:
                want.append(int(server.rng.integers(1, 4000)) if r < 0.7 else 0)      # arrives
            else:
                want.append(0 if r < 0.1 else max(0, n - int(server.rng.integers(1, 9))) if r < 0.25
                            else n if r < 0.3 else min(MAX, n + int(server.rng.integers(1, 500))))
        server.new_inputs(want)
        if graph:
            graph.replay()
        else:
            server.step()
        torch.cuda.synchronize()
        server.check(now, want)
        now = want


def test_index_and_sparse_attention_read_what_was_appended(gpu_lib):
    """The indexer over the appended fp8 keys, and the dense decode over the appended entries."""
    import torch
    server = Server(gpu_lib, 9)
    want = [300, 1000, 17, 2049, 4, 640]
    server.new_inputs(want)
    server.step()
    q = server.rand(B, 32, 64)
    w = torch.rand(B, 32, generator=server.g).cuda()
    scores = gpu_lib.dsa_indexer_scores_fp8(q, w, server.codes, server.scales, server.table, server.lens, MAX)
    keys = server.codes.view(torch.float8_e4m3fn).float().double() * server.scales.double()[..., None]
    for b in range(B):
        t = torch.arange(-(-want[b] // 4), device="cuda")
        k = keys[server.table[b].long()[t // 64], t % 64]
        ref = (torch.relu(k @ q[b].double().T) * w[b].double()).sum(1)
        assert float((scores[b, : len(t)].double() - ref).abs().max() / ref.abs().max()) <= 3e-3
        assert torch.isneginf(scores[b, len(t):]).all()
    # a token that sees the cache alone: the dense decode's
    server.mask.zero_()
    server.counts.fill_(T)
    gpu_lib.dsa_mla_tree_decode(server.q, server.kv, server.table, server.lens, MAX, server.draft, server.mask, SCALE,
                                out=server.out, lse=server.lse, workspace=server.ws)
    for j in (0, T - 1):
        out, lse = gpu_lib.dsa_mla_decode(server.q[:, j].contiguous(), server.kv, server.table, server.lens, MAX, SCALE)
        assert torch.all((lse - server.lse[:, j]).abs() <= 2.0 ** -10 + 2.0 ** -19 * lse.abs())
        assert torch.all((out.float() - server.out[:, j].float()).abs() <= 2.0 ** -6 * out.float().abs().amax())
