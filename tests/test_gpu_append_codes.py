"""GPU tests of dsa_cache_append's 8-bit codes and of rows at the ends of bf16's range.

Codes: they are of u = key * weight against max|u|, as dsa_rmsnorm_fp8's, by the same two-part quotient, so the two entry
points' codes of a key are equal.  Scales: max|u| times the norm's reciprocal over 448; the norms' sums go in
another order (64 squares: up to 2 terms and 5 levels here, 16 terms and 2 levels there, half of their relative error in
the root) and each scale has two or three more roundings: 2^-20 relatively.

Off the exact nearest code: with w = u * 448 / max|u| in fp64 rounded to e4m3 as the reference, a code may differ only
where w lies within the quotient's error of the middle between two codes.  The quotient in two parts is off by under
2^-23 (its last rounding 2^-24, what its parts leave out below that), so |w - middle| <= 2^-22 w there.

Range: y = x * weight / sqrt(mean(x^2) + eps) in fp64; squares of what lies past 2^63 leave fp32, y does not."""
import pytest

pytestmark = pytest.mark.gpu

EPS = 1e-6


def append(lib, keys, weight, eps=EPS):
    import torch
    rows = keys.shape[0]
    pages = -(-rows // 64)
    codes = torch.zeros(pages, 64, 64, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, 64, device="cuda")
    ws = lib.new_workspace(1, 256)
    lib.dsa_cache_append(torch.arange(rows, device="cuda"), index_keys=keys, index_weight=weight, key_codes=codes,
                         key_scales=scales, eps=eps, workspace=ws)
    assert lib.get_error(ws) == 0
    return codes.view(-1, 64)[:rows], scales.view(-1)[:rows]


@pytest.mark.parametrize("w32", [False, True])
@pytest.mark.parametrize("mag", [1.0, 2.0 ** -20, 2.0 ** 20])
def test_codes_are_those_of_the_norm(gpu_lib, w32, mag):
    """A million keys: the same codes from both entry points, and scales within their roundings."""
    import torch
    g = torch.Generator("cuda").manual_seed(5)
    rows = 1 << 20
    keys = (torch.randn(rows, 64, device="cuda", generator=g) * mag).to(torch.bfloat16)
    weight = 1 + 0.3 * torch.randn(64, device="cuda", generator=g)
    weight = weight if w32 else weight.to(torch.bfloat16)
    codes, scales = append(gpu_lib, keys, weight)
    want, want_scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(keys, weight, EPS, 64)
    assert torch.equal(codes, want.view(torch.uint8).view(rows, 64))
    assert not ((scales - want_scales.view(-1)).abs() > 2.0 ** -20 * scales).any()


@pytest.mark.parametrize("norm", [False, True])
def test_codes_against_the_nearest(gpu_lib, norm):
    import torch
    g = torch.Generator("cuda").manual_seed(6)
    rows = 1 << 18
    keys = torch.randn(rows, 64, device="cuda", generator=g).to(torch.bfloat16)
    weight = (1 + 0.3 * torch.randn(64, device="cuda", generator=g)).to(torch.bfloat16) if norm else None
    codes, _ = append(gpu_lib, keys, weight)
    # u in fp32: a product of two bf16 numbers is exact
    u = keys.double() * weight.double() if norm else keys.double()
    w = u * 448 / u.abs().amax(1, keepdim=True)
    values = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()  # 0 to 448
    middles = (values[1:] + values[:-1]) / 2
    got = codes.view(torch.float8_e4m3fn).double().abs()
    at = torch.searchsorted(values, got)
    lo = torch.where(at > 0, middles[(at - 1).clamp(min=0)], torch.full_like(got, -1.0))
    hi = torch.where(at < 126, middles[at.clamp(max=125)], torch.full_like(got, 1e9))
    mag = w.abs()
    assert not ((mag < lo * (1 - 2.0 ** -22)) | (mag > hi * (1 + 2.0 ** -22))).any()
    assert torch.equal(torch.signbit(codes.view(torch.float8_e4m3fn).float()), torch.signbit(u))


@pytest.mark.parametrize("mag, eps", [(2.0 ** 100, EPS), (2.0 ** 124, EPS), (2.0 ** 62, EPS), (2.0 ** -100, 0.0),
                                      (2.0 ** -125, 0.0), (2.0 ** -55, 0.0), (2.0 ** -100, EPS)])
@pytest.mark.parametrize("keys_to", ["fp8", "bf16"])
def test_rows_at_the_ends_of_the_range(gpu_lib, mag, eps, keys_to):
    """Rows whose squares leave fp32 while their norms do not, beside ordinary ones."""
    import torch
    g = torch.Generator("cuda").manual_seed(7)
    rows = 200
    x = torch.randn(rows, 640, device="cuda", generator=g).clamp(-7.9, 7.9)
    x[::2] *= mag
    x[8] = 3.3895e38                                      # bf16's largest number
    x = x.to(torch.bfloat16)
    weight = (1 + 0.3 * torch.randn(640, device="cuda", generator=g)).abs().clamp(min=0.1)
    weight[::3] *= 40
    weight = weight.to(torch.bfloat16)
    pages = 4
    kv = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    to = {"key_pool": torch.zeros(pages, 64, 64, dtype=torch.bfloat16, device="cuda")} if keys_to == "bf16" else {
        "key_codes": torch.zeros(pages, 64, 64, dtype=torch.uint8, device="cuda"),
        "key_scales": torch.zeros(pages, 64, device="cuda")}
    gpu_lib.dsa_cache_append(torch.arange(rows, device="cuda"), latent=x[:, :576], latent_weight=weight[:512].contiguous(),
                             kv_cache=kv, index_keys=x[:, 576:], index_weight=weight[576:].contiguous(), eps=eps, **to)

    def normed(v, w):
        v = v.double()
        return v * w.double() / torch.sqrt((v * v).mean(1, keepdim=True) + eps)

    y = normed(x[:, :512], weight[:512])
    tiny = 2.0 ** -133                                    # half of bf16's last step below its normal numbers
    err = (kv.view(-1, 576)[:rows, :512].double() - y).abs()
    assert not (err > (2.0 ** -8 + 2.0 ** -18) * y.abs() + tiny).any()
    assert torch.isfinite(kv[:3].float()).all()
    y = normed(x[:, 576:], weight[576:])
    if keys_to == "bf16":
        err = (to["key_pool"].view(-1, 64)[:rows].double() - y).abs()
        assert not (err > (2.0 ** -8 + 2.0 ** -18) * y.abs() + tiny).any()
        return
    scales = to["key_scales"].view(-1)[:rows].double()
    top = y.abs().amax(1)
    assert not ((scales - top / 448).abs() > 2.0 ** -18 * top / 448).any()
    got = to["key_codes"].view(-1, 64)[:rows].view(torch.float8_e4m3fn).double() * scales[:, None]
    assert not ((got - y).abs() > 2.0 ** -4 * y.abs() + 2.0 ** -10 * scales[:, None] + 2.0 ** -17 * top[:, None]).any()


@pytest.mark.parametrize("far", ["latent", "key", "both"])
@pytest.mark.parametrize("norm_latent", [True, False])
@pytest.mark.parametrize("keys_to", ["fp8", "bf16"])
def test_one_part_at_the_end_of_the_range(gpu_lib, far, norm_latent, keys_to):
    """Rows of which one part alone is far, with rotation and skipped rows among them, more rows than warps:
    the other part as in ordinary rows, a copied part bit for bit, nothing beside the rows' own entries."""
    import torch
    g = torch.Generator("cuda").manual_seed(8)
    rows, pages = 12000, 200
    x = torch.randn(rows, 640, device="cuda", generator=g)
    which = torch.arange(rows, device="cuda") % 5 == 2
    if far in ("latent", "both"):
        x[which, :512] *= 2.0 ** 90
    if far in ("key", "both"):
        x[which, 576:] *= 2.0 ** 90
    x = x.to(torch.bfloat16)
    slots = torch.randperm(pages * 64, device="cuda", generator=g)[:rows]
    slots[::11] = -1
    weight = (1 + 0.3 * torch.randn(576, device="cuda", generator=g)).to(torch.bfloat16)
    angle = torch.rand(500, 32, device="cuda", generator=g, dtype=torch.float64) * 6
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    positions = torch.randint(500, (rows,), device="cuda", generator=g, dtype=torch.int32)
    kv = torch.full((pages, 64, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    to = {"key_pool": torch.full((pages, 64, 64), 3.0, dtype=torch.bfloat16, device="cuda")} if keys_to == "bf16" else {
        "key_codes": torch.full((pages, 64, 64), 3, dtype=torch.uint8, device="cuda"),
        "key_scales": torch.full((pages, 64), 3.0, device="cuda")}
    gpu_lib.dsa_cache_append(slots, latent=x[:, :576], latent_weight=weight[:512].contiguous() if norm_latent else None,
                             cos_sin=table, positions=positions, kv_cache=kv, index_keys=x[:, 576:],
                             index_weight=weight[512:].contiguous(), eps=EPS, **to)
    live = slots >= 0
    at = slots[live]
    other = torch.ones(pages * 64, dtype=torch.bool, device="cuda")
    other[at] = False
    for t in (kv, *to.values()):
        assert torch.all(t.flatten(0, 1)[other] == 3)

    def normed(v, w):
        v = v.double()
        return v * w.double() / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)

    got = kv.view(-1, 576)[at].double()
    if norm_latent:
        y = normed(x[live, :512], weight[:512])
        assert not ((got[:, :512] - y).abs() > (2.0 ** -8 + 2.0 ** -18) * y.abs()).any()
    else:
        assert torch.equal(kv.view(-1, 576)[at, :512], x[live, :512])
    c, s = table.double()[positions[live].long()].chunk(2, 1)
    a, b = x[live, 512:576:2].double(), x[live, 513:576:2].double()
    for r, want, size in ((got[:, 512::2], a * c - b * s, (a * c).abs() + (b * s).abs()),
                          (got[:, 513::2], a * s + b * c, (a * s).abs() + (b * c).abs())):
        assert not ((r - want).abs() > 2.0 ** -8 * want.abs() + 2.0 ** -22 * size).any()
    y = normed(x[live, 576:], weight[512:])
    if keys_to == "bf16":
        assert not ((to["key_pool"].view(-1, 64)[at].double() - y).abs() > (2.0 ** -8 + 2.0 ** -18) * y.abs()).any()
        return
    scales = to["key_scales"].view(-1)[at].double()
    top = y.abs().amax(1)
    assert not ((scales - top / 448).abs() > 2.0 ** -18 * top / 448).any()
    back = to["key_codes"].view(-1, 64)[at].view(torch.float8_e4m3fn).double() * scales[:, None]
    assert not ((back - y).abs() > 2.0 ** -4 * y.abs() + 2.0 ** -10 * scales[:, None] + 2.0 ** -17 * top[:, None]).any()
