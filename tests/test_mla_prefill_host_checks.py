"""CPU checks of dsa_mla_prefill's argument checks: each rejected call returns its documented status
before any CUDA call; 0 rows launch nothing.  The pointers are plain addresses, never dereferenced."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A, A8, A2 = 0x100000, 0x100008, 0x100002
P = ctypes.c_void_p
I32, I64, SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


@pytest.fixture(scope="module")
def call():
    from sparse_attention_paged_dsa_gb300 import build
    f = ctypes.CDLL(build.build()).dsa_mla_prefill
    f.argtypes = [P, I64, I64, P, I64, I64, P, I64, P, I64, I64, P, P, P, I32, I32, I64, I64, I32, ctypes.c_float, P,
                  P, P, SZ, P]
    f.restype = ctypes.c_int

    def go(**over):
        a = dict(q=A, qr=384, qh=192, kn=A, kr_=512, kh=256, rope=A, rs=576, v=A, vr=512, vh=256, cq=A, ck=A, seq=A,
                 batch=1, heads=2, tq=10, tk=10, e=4, scale=0.1, out=A, lse=A, ws=A, wsb=256)
        a.update(over)
        return f(a["q"], a["qr"], a["qh"], a["kn"], a["kr_"], a["kh"], a["rope"], a["rs"], a["v"], a["vr"], a["vh"],
                 a["cq"], a["ck"], a["seq"], a["batch"], a["heads"], a["tq"], a["tk"], a["e"], a["scale"], a["out"],
                 a["lse"], a["ws"], a["wsb"], None)
    return go


@pytest.mark.parametrize("over, status", [
    (dict(batch=0), INVALID),
    (dict(batch=1025), UNSUPPORTED),
    (dict(heads=0), INVALID),
    (dict(heads=129), UNSUPPORTED),
    (dict(tq=-1), INVALID),
    (dict(tq=1 << 31), UNSUPPORTED),
    (dict(tk=-1), INVALID),
    (dict(tk=1 << 31), UNSUPPORTED),
    (dict(e=0), INVALID),
    (dict(e=65), UNSUPPORTED),
    (dict(scale=-0.1), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID),
    (dict(kn=None), INVALID),
    (dict(rope=None), INVALID),
    (dict(v=None), INVALID),
    (dict(cq=None), INVALID),
    (dict(ck=None), INVALID),
    (dict(seq=None), INVALID),
    (dict(out=None), INVALID),
    (dict(lse=None), INVALID),
    (dict(q=A8), INVALID),
    (dict(kn=A8), INVALID),
    (dict(rope=A8), INVALID),
    (dict(v=A8), INVALID),
    (dict(out=A8), INVALID),
    (dict(lse=A2), INVALID),
    (dict(cq=A2), INVALID),
    (dict(qr=0), INVALID),
    (dict(qh=-192), INVALID),
    (dict(kr_=516), INVALID),                 # not a multiple of 8 elements
    (dict(rs=65), INVALID),
    (dict(vh=1 << 39), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws=A + 64), WORKSPACE),
    (dict(wsb=255), WORKSPACE),
    (dict(tq=0), OK),
    (dict(tq=0, q=None, out=None, lse=None), OK),
])
def test_prefill_rejects_bad_arguments(call, over, status):
    assert call(**over) == status


def test_prefill_workspace_size():
    """More than the error word's header: room for the parts that rows are split into."""
    from sparse_attention_paged_dsa_gb300 import build
    f = ctypes.CDLL(build.build()).dsa_mla_prefill_workspace_size
    f.argtypes, f.restype = [], SZ
    assert f() > 256 + 64 * 512 * 129 * 4
