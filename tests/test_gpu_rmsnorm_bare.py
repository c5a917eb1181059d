"""GPU tests of dsa_rmsnorm_fp8 without a residual, which is dispatched apart (two units a thread above 128
elements), against the formulas in fp64: on each side of every change of the launch, at each alignment, strided and
not, with one scale per 64, 128 elements and row.  Bounds as in test_gpu_rmsnorm.py."""
import pytest
from test_gpu_rmsnorm import EPS, check_bf16, check_codes, reference, rows_of

pytestmark = pytest.mark.gpu

# units of 16 elements: 8 | 9, 32 | 33, 48 | 49, 64 | 65 (a CTA a row behind it), 512 | 513, 1024 | 1025; one element off
# a unit, a multiple of 16 (32-byte rows), of 8 (16-byte rows) and neither
EDGES = [8, 32, 48, 64, 512, 1024]
DIMS = sorted({16 * u + k for u in EDGES for k in (-8, -5, 0, 1, 8, 16)} | {144, 272, 1536, 4096, 7001, 7168, 32768})


@pytest.mark.parametrize("d", DIMS)
def test_norm_fp8_without_a_residual(gpu_lib, d):
    x, w = rows_of(30, 21, d), rows_of(31, 1, d)[0]
    _, y = reference(x, None, w)
    for group in (0, 64, 128):
        codes, scales, out, res = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), EPS, group, with_bf16=True)
        assert res is None
        check_codes(codes, scales, y, group)
        check_bf16(out, y, "out")


@pytest.mark.parametrize("d", [16 * u + k for u in EDGES[:5] for k in (0, 8, 16)] + [7168])
def test_norm_fp8_with_a_residual(gpu_lib, d):
    """The same edges for the rows that have one."""
    x, r, w = rows_of(32, 21, d), rows_of(33, 21, d), rows_of(34, 1, d)[0]
    h, y = reference(x, r, w)
    for group in (0, 64, 128):
        codes, scales, out, res = gpu_lib.dsa_rmsnorm_fp8(x.cuda(), w.cuda(), EPS, group, residual=r.cuda(),
                                                          with_bf16=True)
        check_codes(codes, scales, y, group)
        check_bf16(out, y, "out")
        check_bf16(res, h, "residual_out")


@pytest.mark.parametrize("d, more, start", [(128, 64, 64), (144, 16, 16), (512, 64, 0), (520, 8, 8), (520, 3, 1), (1024, 64, 32),
                                            (1040, 8, 8), (7168, 576, 576), (7168, 3, 2), (8192, 8, 8), (8208, 16, 16)])
def test_norm_fp8_of_strided_rows(gpu_lib, d, more, start):
    """A view of wider rows, on 32-byte, 16-byte and no boundaries; enough rows for the ones fetched ahead."""
    rows = 2500 if d <= 1040 else 700
    wide, w = rows_of(35, rows, d, stride=d + more), rows_of(36, 1, d)[0].float()
    x = wide[:, start:start + d]
    _, y = reference(x, None, w)
    for group in (0, 64, 128):
        codes, scales, out, _ = gpu_lib.dsa_rmsnorm_fp8(wide.cuda()[:, start:start + d], w.cuda(), EPS, group,
                                                        with_bf16=True)
        check_codes(codes, scales, y, group)
        check_bf16(out, y, "out")


@pytest.mark.parametrize("d, offset", [(7, 2), (72, 5), (144, 3), (333, 7), (1000, 4), (1040, 3), (7001, 6), (8192, 1),
                                       (9001, 5), (16403, 2)])
def test_norm_fp8_offset_arrays(gpu_lib, d, offset):
    """Arrays that start anywhere, without a residual: the same values, and nothing beside them."""
    import torch
    rows = 37
    x, w = rows_of(37, rows, d), rows_of(38, 1, d)[0]
    _, y = reference(x, None, w)
    buf = torch.zeros(rows * d + 16, dtype=torch.bfloat16, device="cuda")
    xs = buf[offset:offset + rows * d].view(rows, d).copy_(x)
    ws = torch.cat([w[:1], w]).cuda()[1:]
    for group in (0, 64, 128):
        outs = torch.full((rows * d + 16,), 77.0, dtype=torch.bfloat16, device="cuda")
        cs = torch.full((rows * d + 16,), 0x5A, dtype=torch.uint8, device="cuda")
        a, c = (7 * offset + 2) % 16, (11 * offset + 3) % 16
        out, codes = outs[a:a + rows * d].view(rows, d), cs[c:c + rows * d].view(rows, d)
        _, scales, _, _ = gpu_lib.dsa_rmsnorm_fp8(xs, ws, EPS, group, out=out, codes=codes)
        check_codes(codes, scales, y, group)
        check_bf16(out, y, "out")
        assert torch.all(torch.cat([outs[:a], outs[a + rows * d:]]) == 77.0)
        assert torch.all(torch.cat([cs[:c], cs[c + rows * d:]]) == 0x5A)
