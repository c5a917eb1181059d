"""CPU checks of the argument checks of dsa_pages_update, dsa_cache_append and dsa_mla_tree_decode: each rejected
call returns its documented status before any CUDA call.  The pointers are plain addresses that these paths
never dereference."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A, A8, A4, A2 = 0x100000, 0x100008, 0x100004, 0x100002
P = ctypes.c_void_p
I32, I64, SZ, F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_paged_dsa_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.dsa_pages_update.argtypes = [P, P, I32, I64, P, P, I64, P, I64, P, P, P, P, P, P, SZ, P]
    lib.dsa_cache_append.argtypes = [P, I64, P, I64, P, I32, P, I64, P, P, P, I64, P, I32, P, P, P, I64, F32, P, SZ, P]
    lib.dsa_mla_tree_decode.argtypes = [P, P, I64, P, P, P, P, P, I32, I32, I64, F32, P, P, P, SZ, P]
    lib.dsa_mla_tree_decode_workspace_size.argtypes = [I32, I32]
    lib.dsa_mla_tree_decode_workspace_size.restype = SZ
    return lib


@pytest.mark.parametrize("over, status", [
    (dict(batch=0), INVALID),
    (dict(batch=1025), UNSUPPORTED),
    (dict(ctx=1000), INVALID),
    (dict(ctx=(1 << 24) + 256), UNSUPPORTED),
    (dict(seq=None), INVALID),
    (dict(new=None), INVALID),
    (dict(table=None), INVALID),
    (dict(free=None), INVALID),
    (dict(count=None), INVALID),
    (dict(lens_out=None), INVALID),
    (dict(count_out=None), INVALID),
    (dict(cu=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(pos=None), INVALID),
    (dict(seq=A2), INVALID),
    (dict(table=A2), INVALID),
    (dict(cu=A2), INVALID),
    (dict(slots=A8), INVALID),
    (dict(pos=A8), INVALID),
    (dict(pages=0), INVALID),
    (dict(pages=1 << 31), INVALID),
    (dict(room=-1), INVALID),
    (dict(room=1 << 31), UNSUPPORTED),
    (dict(ws=None), WORKSPACE),
    (dict(ws=A + 16), WORKSPACE),
    (dict(wsb=255), WORKSPACE),
    (dict(room=0, slots=None, pos=None, wsb=0), WORKSPACE),   # no slots: neither array is asked for
])
def test_pages_rejects_bad_arguments(lib, over, status):
    a = dict(seq=A, new=A, batch=2, ctx=8192, table=A, free=A, pages=64, count=A, room=100, lens_out=A, count_out=A, cu=A,
             slots=A, pos=A, ws=A, wsb=256)
    a.update(over)
    assert lib.dsa_pages_update(a["seq"], a["new"], a["batch"], a["ctx"], a["table"], a["free"], a["pages"], a["count"],
                                a["room"], a["lens_out"], a["count_out"], a["cu"], a["slots"], a["pos"], a["ws"],
                                a["wsb"], None) == status


@pytest.mark.parametrize("over, status", [
    (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED),
    (dict(slots=None), INVALID),
    (dict(slots=A4), INVALID),
    (dict(latent=None, keys=None), INVALID),
    (dict(kv=None), INVALID),                          # entries without a cache
    (dict(latent=None), INVALID),                      # a cache without entries
    (dict(latent=None, kv=None, lw=None), INVALID),    # a table without entries
    (dict(latent=None, kv=None, cos=None), INVALID),   # a weight without entries
    (dict(latent=A8), INVALID),
    (dict(kv=A8), INVALID),
    (dict(lstride=580), INVALID),
    (dict(lstride=-576), INVALID),
    (dict(lw=0x100001), INVALID),
    (dict(lw=A2, lw32=1), INVALID),
    (dict(lw32=2), INVALID),
    (dict(cos=A2), INVALID),
    (dict(cos_rows=0), INVALID),
    (dict(pos=None), INVALID),
    (dict(pos=A2), INVALID),
    (dict(keys=None), INVALID),                        # key caches without keys
    (dict(codes=None), INVALID),                       # scales alone
    (dict(scales=None), INVALID),
    (dict(pool=A), INVALID),                           # both formats
    (dict(codes=None, scales=None), INVALID),          # keys without a cache
    (dict(keys=A2), INVALID),
    (dict(kstride=65), INVALID),
    (dict(kstride=-64), INVALID),
    (dict(codes=0x100001), INVALID),
    (dict(scales=A2), INVALID),
    (dict(codes=None, scales=None, pool=A2), INVALID),
    (dict(kw32=-1), INVALID),
    (dict(pages=0), INVALID),
    (dict(pages=1 << 31), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws=A + 64), WORKSPACE),
    (dict(wsb=128), WORKSPACE),
    (dict(rows=0), OK),
    (dict(rows=0, slots=None, latent=None, keys=None, ws=None), OK),
])
def test_append_rejects_bad_arguments(lib, over, status):
    a = dict(slots=A, rows=4, latent=A, lstride=576, lw=A, lw32=0, cos=A, cos_rows=9, pos=A, kv=A, keys=A, kstride=64,
             kw=A, kw32=0, pool=None, codes=A, scales=A, pages=4, eps=1e-6, ws=A, wsb=256)
    a.update(over)
    assert lib.dsa_cache_append(a["slots"], a["rows"], a["latent"], a["lstride"], a["lw"], a["lw32"], a["cos"],
                                a["cos_rows"], a["pos"], a["kv"], a["keys"], a["kstride"], a["kw"], a["kw32"], a["pool"],
                                a["codes"], a["scales"], a["pages"], a["eps"], a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("over, status", [
    (dict(batch=0), INVALID),
    (dict(batch=1025), UNSUPPORTED),
    (dict(tokens=0), INVALID),
    (dict(tokens=65), UNSUPPORTED),
    (dict(ctx=1000), INVALID),
    (dict(ctx=(1 << 24) + 256), UNSUPPORTED),
    (dict(q=None), INVALID),
    (dict(kv=None), INVALID),
    (dict(table=None), INVALID),
    (dict(seq=None), INVALID),
    (dict(draft=None), INVALID),
    (dict(mask=None), INVALID),
    (dict(out=None), INVALID),
    (dict(lse=None), INVALID),
    (dict(q=A8), INVALID),
    (dict(kv=A8), INVALID),
    (dict(draft=A8), INVALID),
    (dict(mask=A4), INVALID),
    (dict(out=A8), INVALID),
    (dict(lse=A2), INVALID),
    (dict(table=A2), INVALID),
    (dict(seq=A2), INVALID),
    (dict(counts=A2), INVALID),
    (dict(pages=0), INVALID),
    (dict(pages=1 << 25), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws=A + 16), WORKSPACE),
    (dict(wsb=128), WORKSPACE),
])
def test_tree_rejects_bad_arguments(lib, over, status):
    a = dict(q=A, kv=A, pages=64, table=A, seq=A, draft=A, mask=A, counts=A, batch=2, tokens=8, ctx=8192, scale=0.1, out=A,
             lse=A, ws=A, wsb=1 << 30)
    a.update(over)
    assert lib.dsa_mla_tree_decode(a["q"], a["kv"], a["pages"], a["table"], a["seq"], a["draft"], a["mask"], a["counts"],
                                   a["batch"], a["tokens"], a["ctx"], a["scale"], a["out"], a["lse"], a["ws"], a["wsb"],
                                   None) == status


def test_tree_workspace_size(lib):
    size = lib.dsa_mla_tree_decode_workspace_size
    assert size(0, 1) == size(1025, 1) == size(4, 0) == size(4, 65) == 0
    for tokens in (1, 2, 3, 8, 27, 64):
        assert 256 < size(1, tokens) == size(1024, tokens) <= 256 << 20


def test_binding_refuses_what_is_not_on_the_gpu():
    """The Python front-end's checks come before the library's."""
    torch = pytest.importorskip("torch")
    from sparse_attention_paged_dsa_gb300 import binding as dsa
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_pages_update(lens, lens, 1024, lens, lens, lens, 4)
    with pytest.raises(TypeError, match="torch.Tensor"):
        dsa.dsa_pages_update([1, 2], lens, 1024, lens, lens, lens, 4)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_cache_append(torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_mla_tree_decode(torch.zeros(1, 2, 64, 576, dtype=torch.bfloat16), None, None, None, 256, None, None, 1.0)
