"""GPU tests of dsa_rmsnorm_fp8 at the ends of fp32's range, against the formulas in fp64.

Below 2^-126 every rounding is of 2^-150 at most: of h * weight (times the norm), of y, and of the scale.  A code is
of y over the scale as stored, so code * scale is within half an e4m3 step of y (2^-4 |y|, 2^-10 scale below normal
codes), or y is past 448 scales; plus the relative errors of test_gpu_rmsnorm.py, 2^-16 of the group's maximum."""
import pytest
from test_gpu_rmsnorm import reference

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -149


def check(codes, scales, x, w, eps, group):
    import torch
    h, y = reference(x, None, w, eps)
    norm = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    vals, scales = codes.cpu().view(torch.float8_e4m3fn).double(), scales.cpu().double()
    assert torch.isfinite(vals).all() and torch.isfinite(scales).all() and (scales > 0).all()
    for i, piece in enumerate(y.split(group or y.shape[1], dim=1)):
        s, amax = scales[:, i:i + 1], piece.abs().amax(1, keepdim=True)
        small = (norm + 2) * ULP
        assert torch.all((s - amax / 448).abs() <= 2.0 ** -17 * amax / 448 + small)
        back = vals[:, i * (group or 0):][:, :piece.shape[1]] * s
        tol = torch.maximum(2.0 ** -4 * piece.abs(), 2.0 ** -10 * s)
        tol = torch.maximum(tol, piece.abs() - 448 * s) + 2.0 ** -16 * amax + small
        err = (back - piece).abs()
        assert not (err > tol).any(), f"{int((err > tol).sum())} codes off, by {float((err / amax).max())} of the maximum"


@pytest.mark.parametrize("group", [0, 64, 128])
@pytest.mark.parametrize("d", [64, 512, 1032, 4096, 7001])
def test_norm_y_past_fp32(gpu_lib, d, group):
    """h * weight is finite, y is not (one element holds the whole row), its scale is."""
    import torch
    x = torch.zeros(3, d, dtype=torch.bfloat16)
    x[0, 5], x[1, d - 1], x[2] = 1.0, -2.0 ** -20, 0.5
    w = torch.full((d,), 3e38)
    codes, scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(x[:2].cuda(), w.cuda(), 1e-18, group)
    for r, (at, value) in enumerate(((5, 3e38 * d ** 0.5), (d - 1, -3e38 * d ** 0.5))):
        vals = codes[r].cpu().view(torch.float8_e4m3fn).double()
        g = at // group if group else 0
        assert torch.isfinite(scales).all() and (scales > 0).all()
        assert abs(vals[at].item() * scales[r, g].item() - value) <= 2.0 ** -4 * abs(value)
        assert int((vals != 0).sum()) == 1


@pytest.mark.parametrize("group", [0, 64, 128])
@pytest.mark.parametrize("d", [64, 512, 1032, 7168])
def test_norm_tiny_products(gpu_lib, d, group):
    """h * weight below 2^-126, but scaled back up by the norm: scales are ordinary numbers."""
    import torch
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(5, d, generator=g) * 2.0 ** -32).to(torch.bfloat16)
    for value in (1e-30, 1e-32, 1e-33):
        w = (torch.rand(d, generator=g) + 0.5) * value
        codes, scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), 1e-24, group)
        check(codes, scales, x, w, 1e-24, group)


@pytest.mark.parametrize("group", [0, 64, 128])
@pytest.mark.parametrize("d", [64, 512, 1032, 7168])
def test_norm_tiny_scales(gpu_lib, d, group):
    """Scales below 2^-126, down to a few steps of 2^-149: the codes go by the scale as it is stored."""
    import torch
    g = torch.Generator().manual_seed(d + 1)
    x = (torch.randn(16, d, generator=g) * torch.exp(torch.randn(16, 1, generator=g))).to(torch.bfloat16)
    for value in (1e-36, 1e-38, 1e-40, 1e-41, 3e-42):
        w = torch.full((d,), value)
        codes, scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), 1e-6, group)
        check(codes, scales, x, w, 1e-6, group)


@pytest.mark.parametrize("group", [0, 64, 128])
def test_norm_vanishing_squares(gpu_lib, group):
    """Squares below fp32's range with eps = 0: no finite norm, but scales that an index-key cache may hold."""
    import torch
    x = torch.full((4, 256), 1e-30, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 7:] = 0
    _, scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), torch.ones(256).cuda(), 0.0, group)
    assert torch.isfinite(scales).all() and (scales > 0).all()
