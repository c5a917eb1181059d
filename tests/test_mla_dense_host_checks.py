"""CPU checks of dsa_mla_decode's argument checks: each rejected call returns its documented status
before any CUDA call.  The pointers are plain addresses that these paths never dereference."""
import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
A, A8, A4 = 0x100000, 0x100008, 0x100002
P = ctypes.c_void_p
I32, I64, SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_paged_dsa_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.dsa_mla_decode.argtypes = [P, P, I64, P, P, I32, I32, I64, ctypes.c_float, P, P, P, SZ, P]
    lib.dsa_mla_decode.restype = ctypes.c_int
    lib.dsa_mla_decode_workspace_size.argtypes = [I32, I32]
    lib.dsa_mla_decode_workspace_size.restype = SZ
    return lib


@pytest.mark.parametrize("over, status", [
    (dict(batch=0), INVALID),
    (dict(batch=1025), UNSUPPORTED),
    (dict(next_n=0), INVALID),
    (dict(next_n=5), INVALID),
    (dict(ctx=1000), INVALID),
    (dict(ctx=(1 << 24) + 256), UNSUPPORTED),
    (dict(q=None), INVALID),
    (dict(kv=None), INVALID),
    (dict(table=None), INVALID),
    (dict(seq=None), INVALID),
    (dict(out=None), INVALID),
    (dict(lse=None), INVALID),
    (dict(q=A8), INVALID),
    (dict(kv=A8), INVALID),
    (dict(out=A8), INVALID),
    (dict(lse=A8), INVALID),
    (dict(table=A4), INVALID),
    (dict(seq=A4), INVALID),
    (dict(pages=0), INVALID),
    (dict(pages=1 << 25), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws=A + 16), WORKSPACE),
    (dict(wsb=128), WORKSPACE),
])
def test_decode_rejects_bad_arguments(lib, over, status):
    a = dict(q=A, kv=A, pages=64, table=A, seq=A, batch=2, next_n=1, ctx=8192, scale=0.1, out=A, lse=A, ws=A,
             wsb=1 << 30)
    a.update(over)
    assert lib.dsa_mla_decode(a["q"], a["kv"], a["pages"], a["table"], a["seq"], a["batch"], a["next_n"], a["ctx"],
                              a["scale"], a["out"], a["lse"], a["ws"], a["wsb"], None) == status


def test_decode_workspace_size(lib):
    size = lib.dsa_mla_decode_workspace_size
    assert size(0, 1) == size(1025, 1) == size(4, 0) == size(4, 5) == 0
    assert 256 < size(1, 1) <= 64 << 20 and size(1, 1) == size(1024, 1)
