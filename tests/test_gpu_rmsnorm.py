"""GPU tests of dsa_rmsnorm / dsa_rmsnorm_fp8 against the same formulas in fp64.

Tolerances from the arithmetic (u = 2^-24, fp32 half step).  h = x + r is one fp32 rounding of
exact bf16 inputs.  The sum of squares adds at most 32 terms per thread, 10 butterfly levels and
the square's own rounding: below 45 u relatively, halved by the root, plus rsqrtf (2 ulp = 4 u),
the division by d, + eps and the two products of y: |y32 - y| < 34 u |y| < 2^-18 |y|.
  bf16 outputs: one half step on top, (2^-8 + 2^-17) |y|;
  scales: the same relative error plus one division: 2^-17;
  codes: code * scale is within half an e4m3 step of y (2^-4 |y| for normal codes, 2^-10 scale
  below them) plus the errors of y and scale, 2^-16 of the group's maximum."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

EPS = 1e-6


def rows_of(seed, rows, d, stride=None, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, stride or d, generator=g, dtype=torch.float32) * scale
    x *= torch.exp(torch.randn(rows, 1, generator=g))
    return x.to(torch.bfloat16)


def reference(x, residual, weight, eps=EPS):
    import torch
    h = x.double() + (residual.double() if residual is not None else 0)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * weight.double()
    return h, y


def check_bf16(got, want, what):
    bad = (got.double().cpu() - want).abs() > (2.0 ** -8 + 2.0 ** -17) * want.abs() + 1e-38
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, first at {bad.nonzero()[0].tolist()}"


def check_codes(codes, scales, y, group):
    import torch
    rows, d = y.shape
    g = group or d
    vals = codes.cpu().view(torch.float8_e4m3fn).double()
    scales = scales.cpu().double()
    for i, piece in enumerate(y.split(g, dim=1)):
        amax = piece.abs().amax(1)
        want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        s = scales[:, i]
        assert torch.all((s - want).abs() <= 2.0 ** -17 * want)
        err = (vals[:, i * g:i * g + piece.shape[1]] * s[:, None] - piece).abs()
        tol = torch.maximum(2.0 ** -4 * piece.abs(), 2.0 ** -10 * s[:, None]) + 2.0 ** -16 * amax[:, None]
        assert not (err > tol).any()


SHAPES = [(1, 1), (3, 7), (5, 8), (33, 63), (40, 64), (2, 65), (17, 120), (300, 128), (9, 129), (7, 256), (31, 264),
          (1, 512), (4099, 512), (12, 513), (5, 1000), (3, 1024), (3, 1032), (2, 4104), (1, 7168), (64, 7168),
          (700, 7168), (2, 8192), (2, 8200), (620, 8200), (1, 16384), (2, 16392), (3, 32761), (700, 16400), (2, 32768)]


@pytest.mark.parametrize("rows, d", SHAPES)
def test_norm_bf16(gpu_lib, rows, d):
    import torch
    x, r = rows_of(1, rows, d), rows_of(2, rows, d, scale=3.0)
    w = rows_of(3, 1, d)[0]
    for residual in (r, None):
        h, y = reference(x, residual, w)
        out, res_out = gpu_lib.dsa_rmsnorm(x.cuda(), w.cuda(), EPS,
                                           residual=None if residual is None else residual.cuda())
        check_bf16(out, y, "out")
        if residual is None:
            assert res_out is None
        else:
            assert torch.equal(res_out.cpu(), (x.float() + r.float()).to(torch.bfloat16))


@pytest.mark.parametrize("group", [0, 64, 128])
@pytest.mark.parametrize("rows, d", SHAPES)
def test_norm_fp8(gpu_lib, rows, d, group):
    x, r = rows_of(4, rows, d), rows_of(5, rows, d)
    w = rows_of(6, 1, d)[0].float()
    h, y = reference(x, r, w)
    codes, scales, out, res_out = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), EPS, group, residual=r.cuda(),
                                                          with_bf16=True)
    check_codes(codes, scales, y, group)
    check_bf16(out, y, "out")
    check_bf16(res_out, h, "residual_out")
    again = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), EPS, group, residual=r.cuda())
    assert again[2] is None and np.array_equal(again[0].view(__import__("torch").uint8).cpu().numpy(),
                                               codes.view(__import__("torch").uint8).cpu().numpy())


@pytest.mark.parametrize("d, stride", [(512, 576), (512, 515), (64, 72), (7168, 7171), (100, 104)])
def test_norm_strided_rows(gpu_lib, d, stride):
    wide = rows_of(7, 77, d, stride=stride)
    w = rows_of(8, 1, d)[0]
    for start in (0, 1, 3):
        if start + d > stride:
            continue
        x = wide[:, start:start + d]
        out, _ = gpu_lib.dsa_rmsnorm(wide.cuda()[:, start:start + d], w.cuda(), EPS)
        check_bf16(out, reference(x, None, w)[1], f"start {start}")


@pytest.mark.parametrize("d, offset", [(1, 1), (7, 2), (24, 1), (65, 3), (72, 5), (333, 7), (1000, 4), (1037, 1), (1040, 3),
                                       (7001, 6), (8192, 1), (9001, 5), (16403, 2)])
def test_norm_offset_arrays(gpu_lib, d, offset):
    """Arrays that start anywhere, each at its own offset: the same values, and nothing beside them."""
    import torch
    rows = 37
    x, r, w = rows_of(24, rows, d), rows_of(25, rows, d, scale=2.0), rows_of(26, 1, d)[0]
    h, y = reference(x, r, w)
    u8 = torch.uint8
    buffers = {}

    def at(name, k, data=None, dtype=torch.bfloat16):
        buf = torch.full((rows * d + 64,), 0x5A, dtype=u8, device="cuda").to(dtype) if dtype is u8 else \
            torch.full((rows * d + 64,), 77.0, dtype=dtype, device="cuda")
        buffers[name] = (buf, k, rows * d)
        view = buf[k:k + rows * d].view(rows, d)
        if data is not None:
            view.copy_(data)
        return view

    args = at("x", offset, x), torch.cat([w[:1], w]).cuda()[1:], EPS
    kw = dict(residual=at("r", (3 * offset) % 16, r), residual_out=at("ro", (5 * offset + 1) % 16))
    for group in (-1, 0, 64, 128):
        out = at("out", (7 * offset + 2) % 16)
        if group < 0:
            gpu_lib.dsa_rmsnorm(*args, out=out, **kw)
        else:
            codes = at("codes", (11 * offset + 3) % 16, dtype=u8)
            _, scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(*args, group, out=out, codes=codes, **kw)
            check_codes(codes, scales, y, group)
        check_bf16(out, y, "out")
        assert torch.equal(kw["residual_out"].cpu(), (x.float() + r.float()).to(torch.bfloat16))
        for name, (buf, k, n) in buffers.items():
            beside = torch.cat([buf[:k], buf[k + n:]])
            assert torch.all(beside == (0x5A if buf.dtype is u8 else 77.0)), name


def test_norm_broadcast_row(gpu_lib):
    """Stride 0: the same row every time."""
    x, w = rows_of(9, 1, 640), rows_of(10, 1, 640)[0]
    out, _ = gpu_lib.dsa_rmsnorm(x.cuda().expand(50, 640), w.cuda(), EPS)
    check_bf16(out, reference(x.expand(50, 640), None, w)[1], "out")


@pytest.mark.parametrize("d", [100, 512, 7168])
def test_norm_in_place(gpu_lib, d):
    """out on x and residual_out on residual, as a decoder layer keeps its stream."""
    x, r, w = rows_of(11, 65, d), rows_of(12, 65, d), rows_of(13, 1, d)[0]
    h, y = reference(x, r, w)
    xd, rd = x.cuda(), r.cuda()
    out, res = gpu_lib.dsa_rmsnorm(xd, w.cuda(), EPS, residual=rd, out=xd, residual_out=rd)
    assert out.data_ptr() == xd.data_ptr() and res.data_ptr() == rd.data_ptr()
    check_bf16(xd, y, "out")
    check_bf16(rd, h, "residual_out")


def test_norm_zero_and_tiny_rows(gpu_lib):
    """A zero row, a row of fp32-tiny results (scales below 2^-126) and one that fp32 cannot scale."""
    import torch
    d = 128
    x = torch.zeros(4, d, dtype=torch.bfloat16)
    x[1, 5] = 1.0
    x[2] = rows_of(14, 1, d)[0]
    x[3] = rows_of(15, 1, d)[0]
    w = torch.ones(d)
    for value in (1.0, 1e-36, 1e-42):
        codes, scales, out, _ = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), (w * value).cuda(), EPS, 128, with_bf16=True)
        vals = codes.cpu().view(torch.float8_e4m3fn).double()
        assert torch.isfinite(vals).all() and torch.isfinite(scales).all() and (scales > 0).all()
        assert scales[0].item() == 1.0 and not vals[0].any() and not out[0].any()
        if value > 1e-40:
            # scale has at least 2^-149 steps: 1e-36 / 448 is 2^-128.4, held to 2^-21 relatively
            y = reference(x, None, (w * value))[1]
            back = vals * scales.cpu().double()
            tol = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * scales.cpu().double()) + 2.0 ** -16 * y.abs().amax(
                1, keepdim=True)
            assert torch.all((back - y).abs() <= tol)


def test_norm_non_finite_rows_stay_alone(gpu_lib):
    """A NaN or infinite element reaches its own row's outputs only."""
    import torch
    for d in (64, 512, 7168):
        x, w = rows_of(16, 40, d), rows_of(17, 1, d)[0]
        bad = x.clone()
        bad[3, d // 2] = float("nan")
        bad[8, 0] = float("inf")
        good = [i for i in range(40) if i not in (3, 8)]
        a = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), EPS, 64, with_bf16=True)
        b = gpu_lib.dsa_rmsnorm_fp8(bad.cuda(), w.cuda(), EPS, 64, with_bf16=True)
        for p, q in zip(a[:3], b[:3]):
            p, q = p.view(torch.uint8).cpu(), q.view(torch.uint8).cpu()
            assert torch.equal(p[good], q[good])
        assert torch.isnan(b[2][3].float()).all()


def test_norm_index_keys(gpu_lib, oracle):
    """Rows of 64 with group 64 are an fp8 index-key cache: the indexer scores them as they stand for."""
    import torch
    from sparse_attention_paged_dsa_gb300 import inputs as I
    case = I.make_case(name="keys", batch=2, max_context=8192, seq_lens=[8192, 700], num_pages=48, k=64, seed=5)
    q, w, pool, table, seq = gpu_lib.to_device(case)
    weight = rows_of(18, 1, 64)[0].cuda()
    codes, scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(pool.view(-1, 64), weight, EPS, 64)
    codes, scales = codes.view(-1, 64, 64), scales.view(-1, 64)
    got = gpu_lib.dsa_indexer_scores_fp8(q, w, codes, scales, table, seq, case.max_context).cpu().numpy()
    f = I.with_fp8_keys(case)
    f.key_codes, f.key_scales = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    want = oracle.case_scores_fp8(f)
    for b, n in enumerate(case.live_positions()):
        assert np.abs(got[b, :n] - want[b, :n]).max() <= 3e-3 * np.abs(want[b, :n]).max()


def test_norm_streams_and_graph(gpu_lib):
    """On a side stream, and captured and replayed on new values: the same bits as a plain call."""
    import torch
    x, r, w = rows_of(19, 64, 7168).cuda(), rows_of(20, 64, 7168).cuda(), rows_of(21, 1, 7168)[0].cuda()
    want = [t.clone() for t in gpu_lib.dsa_rmsnorm(x, w, EPS, residual=r)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gpu_lib.dsa_rmsnorm(x, w, EPS, residual=r)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out, res = torch.empty_like(x), torch.empty_like(x)
    xs = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.dsa_rmsnorm(xs, w, EPS, residual=r, out=out, residual_out=res)
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(res, want[1])


def test_norm_refusals(gpu_lib):
    import torch
    x, w = rows_of(22, 4, 64).cuda(), rows_of(23, 1, 64)[0].cuda()
    with pytest.raises(ValueError):
        gpu_lib.dsa_rmsnorm(x.cpu(), w, EPS)
    with pytest.raises(TypeError):
        gpu_lib.dsa_rmsnorm(x.float(), w, EPS)
    with pytest.raises(ValueError):
        gpu_lib.dsa_rmsnorm(x, w[:32], EPS)
    with pytest.raises(ValueError):
        gpu_lib.dsa_rmsnorm(x.t(), rows_of(23, 1, 4)[0].cuda(), EPS)
    with pytest.raises(ValueError):
        gpu_lib.dsa_rmsnorm(x, w, EPS, residual=x[:3])
    with pytest.raises(ValueError):
        gpu_lib.dsa_rmsnorm(x, w, EPS, residual_out=x.clone())
    with pytest.raises(ValueError):
        gpu_lib.dsa_rmsnorm_fp8(x, w, EPS, 32)
    with pytest.raises(gpu_lib.DsaError):
        gpu_lib.dsa_rmsnorm(x, w, float("nan"))
    with pytest.raises(gpu_lib.DsaError):  # out must not be residual_out
        y = x.clone()
        gpu_lib.dsa_rmsnorm(x, w, EPS, residual=x, out=y, residual_out=y)
    empty, none = gpu_lib.dsa_rmsnorm(x[:0], w, EPS)
    assert empty.shape == (0, 64) and none is None
