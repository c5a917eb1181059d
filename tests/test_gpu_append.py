"""GPU tests of dsa_cache_append against the same formulas in fp64.

Tolerances from the arithmetic (u = 2^-24, fp32 half step).  Norms: the sum of 512 squares adds at most
16 terms a lane and 5 butterfly levels, with the square's own rounding below 22 u relatively, halved by
the root; + eps, the reciprocal root (2 ulp, 4 u) and two products add 7 u: |y32 - y| < 18 u |y| <
2^-19 |y|.  bf16 outputs: half a step on top, (2^-8 + 2^-18) |y|.  Rotation: two products and a sum, 3 u
(|a c| + |b s|) before the rounding to bf16.  Scales: 2^-18 relatively.  Codes: within half an e4m3 step
(2^-4 |y| for normal codes, 2^-10 scale below them) plus the errors of y and scale, 2^-17 of the largest."""
import pytest

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Case:
    def __init__(self, rows, pages, seed=1, latent=True, norm=True, rope=True, keys="fp8", w32=False, wide=0, mag=1.0):
        import torch
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        bf = lambda t: t.to(torch.bfloat16).cuda()  # noqa: E731
        self.keys_to, self.norm = keys, norm
        product = bf(rand(rows, 576 + 64 + wide) * torch.exp(rand(rows, 1)) * mag)
        slots = torch.randperm(pages * 64, generator=g)[:rows]
        if rows > 2:
            slots[::7] = -1
        self.slots = slots.cuda()
        self.kw = {}
        if latent:
            self.kw.update(latent=product[:, :576] if wide else product[:, :576].contiguous(), kv_cache=bf(rand(pages, 64, 576)))
            if norm:
                self.kw["latent_weight"] = (1 + 0.3 * rand(512)).cuda() if w32 else bf(1 + 0.3 * rand(512))
            if rope:
                angle = rand(1000, 32).double() * 100
                self.kw["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
                self.kw["positions"] = torch.randint(1000, (rows,), generator=g).to(torch.int32).cuda()
        if keys:
            k = product[:, 576:640]
            self.kw["index_keys"] = k if wide else k.contiguous()
            if norm:
                self.kw["index_weight"] = (1 + 0.3 * rand(64)).cuda() if w32 else bf(1 + 0.3 * rand(64))
            if keys == "bf16":
                self.kw["key_pool"] = bf(rand(pages, 64, 64))
            else:
                self.kw["key_codes"] = torch.randint(256, (pages, 64, 64), generator=g, dtype=torch.uint8).cuda()
                self.kw["key_scales"] = rand(pages, 64).cuda()
        self.before = {k: v.clone() for k, v in self.kw.items() if k in ("kv_cache", "key_pool", "key_codes", "key_scales")}

    def run(self, lib, error=0, **over):
        ws = lib.new_workspace(1, 256)
        lib.dsa_cache_append(self.slots, **dict(self.kw, **over), eps=EPS, workspace=ws)
        assert lib.get_error(ws) == error

    def check(self, skip=()):
        """All caches: the written entries within their bounds, every other byte as it was."""
        import torch
        rows = torch.tensor([i for i, s in enumerate(self.slots.tolist()) if s != -1 and i not in skip], dtype=torch.int64,
                            device="cuda")
        to = self.slots[rows]
        normed = lambda x, w: x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w.double()  # noqa: E731
        for name, was in self.before.items():
            now = self.kw[name].flatten(0, 1)
            other = torch.ones(now.shape[0], dtype=torch.bool, device="cuda")
            other[to] = False
            a, b = now[other], was.flatten(0, 1)[other]
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"{name}: other entries changed"
        if "latent" in self.kw:
            x = self.kw["latent"][rows].double()
            got = self.kw["kv_cache"].view(-1, 576)[to].double()
            y = normed(x[:, :512], self.kw["latent_weight"]) if "latent_weight" in self.kw else x[:, :512]
            exact = "latent_weight" not in self.kw
            assert not ((got[:, :512] - y).abs() > (0 if exact else 2.0 ** -8 + 2.0 ** -18) * y.abs() + 0).any()
            r = x[:, 512:]
            if "cos_sin" in self.kw:
                c, s = self.kw["cos_sin"].double()[self.kw["positions"][rows].long()].chunk(2, 1)
                a, b = r[:, 0::2], r[:, 1::2]
                for got_p, want, size in ((got[:, 512::2], a * c - b * s, (a * c).abs() + (b * s).abs()),
                                          (got[:, 513::2], a * s + b * c, (a * s).abs() + (b * c).abs())):
                    assert not ((got_p - want).abs() > 2.0 ** -8 * want.abs() + 2.0 ** -22 * size).any()
            else:
                assert torch.equal(got[:, 512:], r)
        if "index_keys" not in self.kw:
            return
        k = self.kw["index_keys"][rows].double()
        y = normed(k, self.kw["index_weight"]) if "index_weight" in self.kw else k
        if self.keys_to == "bf16":
            got = self.kw["key_pool"].view(-1, 64)[to].double()
            assert not ((got - y).abs() > (2.0 ** -8 + 2.0 ** -18 if "index_weight" in self.kw else 0) * y.abs()).any()
            return
        codes = self.kw["key_codes"].view(-1, 64)[to].view(torch.float8_e4m3fn).float().double()
        scales = self.kw["key_scales"].view(-1)[to].double()
        top = y.abs().amax(1)
        want = torch.where(top > 0, top / 448, torch.ones_like(top))
        assert not ((scales - want).abs() > 2.0 ** -18 * want).any()
        err = (codes * scales[:, None] - y).abs()
        assert not (err > 2.0 ** -4 * y.abs() + 2.0 ** -10 * scales[:, None] + 2.0 ** -17 * top[:, None]).any()


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 63, 64, 65, 300, 4099])
def test_append_rows(gpu_lib, rows):
    case = Case(rows, rows // 64 + 2, seed=rows)
    case.run(gpu_lib)
    case.check()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("keys", [None, "bf16", "fp8"])
@pytest.mark.parametrize("wide", [0, 8, 56])
def test_append_parts(gpu_lib, norm, rope, keys, wide):
    """Each part with and without its computation, on rows of their own and as views of a wide product."""
    case = Case(101, 4, seed=wide, norm=norm, rope=rope, keys=keys, wide=wide, w32=wide == 8)
    case.run(gpu_lib)
    case.check()


@pytest.mark.parametrize("keys", ["bf16", "fp8"])
@pytest.mark.parametrize("norm", [False, True])
def test_append_index_keys_alone(gpu_lib, keys, norm):
    """Keys alone; rows a pair of elements apart from 4-byte boundaries."""
    case = Case(77, 3, latent=False, norm=norm, keys=keys, wide=2, seed=3)
    case.run(gpu_lib)
    case.check()


def test_append_many(gpu_lib):
    """More rows than the device holds at a time."""
    case = Case(60001, 1200, seed=5, wide=24)
    case.run(gpu_lib)
    case.check()


def test_append_small_and_large_values(gpu_lib):
    for mag in (2.0 ** -30, 2.0 ** 30):
        case = Case(65, 3, seed=6, mag=mag)
        case.run(gpu_lib)
        case.check()


def test_append_zero_and_non_finite_keys(gpu_lib):
    """A key of zeros has scale 1 and codes 0; one without a finite scale has scale 1: every scale is positive."""
    import torch
    case = Case(6, 2, norm=False, keys="fp8", seed=7)
    case.slots.copy_(torch.arange(6))
    keys = case.kw["index_keys"]
    keys[0] = 0
    keys[1, 5] = float("inf")
    keys[2, 5] = float("nan")
    keys[3] = 1e-40
    case.run(gpu_lib)
    scales, codes = case.kw["key_scales"].view(-1), case.kw["key_codes"].view(-1, 64)
    assert scales[0] == 1 and not codes[0].any()
    assert scales[1] == 1 and codes[1, 5] == 0x7E
    assert torch.isfinite(scales[:6]).all() and (scales[:6] > 0).all()
    assert codes[2, 5] & 0x7F == 0x7F


def test_append_bad_slots_and_positions(gpu_lib):
    """Rows whose slot or position is out of range are left out and flagged."""
    case = Case(50, 2, seed=8)
    case.slots[3], case.slots[4], case.slots[20] = 128, -2, 1 << 40
    case.run(gpu_lib, error=gpu_lib.DEVERR_BAD_PAGE)
    case.check(skip=(3, 4, 20))
    case = Case(50, 2, seed=9)
    case.kw["positions"][5], case.kw["positions"][6] = 1000, -1
    case.slots[5], case.slots[6] = 120, 121
    case.slots[(case.slots == 120) | (case.slots == 121)] = -1
    case.slots[5], case.slots[6] = 120, 121
    case.run(gpu_lib, error=gpu_lib.DEVERR_BAD_RANGE)
    case.check(skip=(5, 6))


def test_append_skips_all_and_nothing(gpu_lib):
    import torch
    case = Case(9, 2, seed=10)
    case.slots.fill_(-1)
    case.run(gpu_lib)
    case.check()
    empty = Case(9, 2, seed=11)
    empty.slots = torch.empty(0, dtype=torch.int64, device="cuda")
    for k in ("latent", "index_keys", "positions"):
        empty.kw[k] = empty.kw[k][:0]
    empty.run(gpu_lib)
    empty.check()


def test_append_far_slots(gpu_lib):
    """Slots whose elements lie past 2^31 in the cache."""
    import torch
    pages = 60000                                                     # 2.2 G elements, 4.4 GB
    case = Case(40, 2, keys="bf16", seed=12)
    case.kw["kv_cache"] = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    case.kw["key_pool"] = torch.zeros(pages, 64, 64, dtype=torch.bfloat16, device="cuda")
    near = case.slots.clone()
    case.slots = torch.where(near >= 0, near + (pages - 2) * 64, near)
    case.run(gpu_lib)
    assert not case.kw["kv_cache"][: pages - 2].any()
    case.kw["kv_cache"], case.kw["key_pool"] = case.kw["kv_cache"][-2:].clone(), case.kw["key_pool"][-2:].clone()
    case.before = {k: torch.zeros_like(case.kw[k]) for k in ("kv_cache", "key_pool")}
    case.slots = near
    case.check()


def test_append_graph(gpu_lib):
    """One capture, replayed with other slots and rows; both outputs the same bits as an eager call's."""
    import torch
    case = Case(200, 8, seed=13)
    other = Case(200, 8, seed=14)
    ws = gpu_lib.new_workspace(1, 256)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu_lib.dsa_cache_append(case.slots, **case.kw, eps=EPS, workspace=ws)
    graph.replay()
    case.check()
    for k in ("latent", "index_keys", "positions"):
        case.kw[k].copy_(other.kw[k])
    case.slots.copy_(other.slots)
    case.before = {k: case.kw[k].clone() for k in case.before}
    graph.replay()
    case.check()
    assert gpu_lib.get_error(ws) == 0
