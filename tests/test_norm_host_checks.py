"""CPU checks of the RMS norm entry points' argument checks: every rejected call returns the status
include/dsa_indexer.h documents before any CUDA call, and rows = 0 launches nothing.  The pointers
are plain addresses that these paths never dereference."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
A, B, C, D, E = (0x100000 * (i + 1) for i in range(5))
P = ctypes.c_void_p
I32, I64, F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_paged_dsa_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.dsa_rmsnorm.argtypes = [P, I64, P, P, I32, I64, I32, F32, P, P, P]
    lib.dsa_rmsnorm_fp8.argtypes = [P, I64, P, P, I32, I64, I32, F32, I32, P, P, P, P, P]
    lib.dsa_rmsnorm.restype = lib.dsa_rmsnorm_fp8.restype = ctypes.c_int
    return lib


def call(lib, fp8, **over):
    a = dict(x=A, stride=512, res=B, w=C, w32=0, rows=4, d=512, eps=1e-6, group=128, res_out=B, out=D, codes=E,
             scales=E + 0x1000)
    a.update(over)
    head = [a["x"], a["stride"], a["res"], a["w"], a["w32"], a["rows"], a["d"], a["eps"]]
    if fp8:
        return lib.dsa_rmsnorm_fp8(*head, a["group"], a["res_out"], a["out"], a["codes"], a["scales"], None)
    return lib.dsa_rmsnorm(*head, a["res_out"], a["out"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("over, status", [
    (dict(x=None), INVALID),
    (dict(w=None), INVALID),
    (dict(x=A + 1), INVALID),                       # not on an element's boundary
    (dict(w=C + 2, w32=1), INVALID),
    (dict(w32=2), INVALID),
    (dict(res=None), INVALID),                      # residual_out without a residual
    (dict(res_out=None), INVALID),                  # a residual without residual_out
    (dict(stride=-512), INVALID),
    (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), INVALID),
    (dict(d=0), INVALID),
    (dict(d=32769), UNSUPPORTED),
    (dict(eps=-1e-6), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(out=B), INVALID),                         # out is residual_out
    (dict(out=A, stride=576), INVALID),             # in place on strided rows
    (dict(res_out=A, stride=0), INVALID),
    (dict(rows=0), OK),
    (dict(rows=0, x=None, res=None, w=None, res_out=None, out=None), OK),
])
def test_norm_rejects_bad_arguments(lib, fp8, over, status):
    assert call(lib, fp8, **over) == status


@pytest.mark.parametrize("over", [dict(group=32), dict(group=-1), dict(group=512), dict(codes=None),
                                  dict(scales=None), dict(scales=E + 2)])
def test_norm_fp8_rejects_bad_arguments(lib, over):
    assert call(lib, True, **over) == INVALID


def test_norm_needs_an_output(lib):
    assert call(lib, False, out=None) == INVALID
