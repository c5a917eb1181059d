"""GPU tests of the latent attentions on values that their contract leaves out but a caller has to be able to
find: a NaN or an infinity among what a row sees reaches that row's output and its lse, split or not, as the
formulas in fp64 have it, and no other row."""
import pytest
from test_gpu_mla_decode import Case as Decode
from test_gpu_mla_prefill import Case as Prefill

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def same_kind(out, lse, o, l, what):
    """out is NaN just where the formulas in fp64 have it; lse where theirs is NaN or, from an infinite score, +inf."""
    import torch
    assert torch.equal(torch.isnan(out), torch.isnan(o)), f"{what}: out"
    assert torch.equal(torch.isnan(lse), torch.isnan(l) | torch.isposinf(l)), f"{what}: lse"
    assert torch.equal(torch.isneginf(lse), torch.isneginf(l)), f"{what}: lse of nothing seen"
    assert not torch.isinf(out).any() and not torch.isposinf(lse).any(), what


# one request over every SM; one that is never cut; 200, of which a range holds several, whole and in parts
@pytest.mark.parametrize("seqs, context, rows", [([20000], 20480, [0]), ([1000, 60], 1024, [0, 1]),
                                                 ([2000 + b for b in range(200)], 2304, [0, 57, 101, 199])])
@pytest.mark.parametrize("dim, value", [(3, NAN), (540, NAN), (540, INF), (540, -INF)])
def test_decode_entry_that_is_seen(gpu_lib, seqs, context, rows, dim, value):
    import torch
    case = Decode(seqs, context, next_n=2, seed=60)
    ws = gpu_lib.new_mla_workspace(len(seqs), 2)
    want = [t.clone() for t in gpu_lib.dsa_mla_decode(*case.args(), workspace=ws)]
    for b in rows:
        t = case.live(b, 0) // 3
        case.kv[case.table[b, t // 64].long(), t % 64, dim] = value
    out, lse = gpu_lib.dsa_mla_decode(*case.args(), workspace=ws)
    for b in range(len(seqs)):
        if b not in rows:
            assert torch.equal(out[b], want[0][b]) and torch.equal(lse[b], want[1][b]), b
            continue
        for j in range(2):
            o, l, _ = case.reference(b, j)
            same_kind(out[b, j], lse[b, j], o, l, f"request {b} token {j}")
    assert torch.isnan(lse[rows]).any()
    assert gpu_lib.get_error(ws) == 0


@pytest.mark.parametrize("seqs, context", [([20000], 20480), ([1000, 60], 1024)])
def test_decode_head_of_q(gpu_lib, seqs, context):
    import torch
    case = Decode(seqs, context, seed=61)
    ws = gpu_lib.new_mla_workspace(len(seqs))
    want = [t.clone() for t in gpu_lib.dsa_mla_decode(*case.args(), workspace=ws)]
    case.q[0, 0, 37, 100] = NAN
    out, lse = gpu_lib.dsa_mla_decode(*case.args(), workspace=ws)
    assert torch.isnan(out[0, 0, 37]).all() and torch.isnan(lse[0, 0, 37])
    for t, w in ((out, want[0]), (lse, want[1])):
        t[0, 0, 37] = w[0, 0, 37]
        assert torch.equal(t, w)


# one tile; several tiles and blocks; in parts: one row, both kinds of unit, several requests
@pytest.mark.parametrize("new, seqs, heads, split", [([100], [100], 2, False), ([700, 200], [1500, 200], 3, False),
                                                     ([1], [9999], 1, True), ([130], [20000], 3, True),
                                                     ([600], [12000], 4, True), ([40, 9], [20000, 5000], 3, True)])
@pytest.mark.parametrize("where, value", [("key", NAN), ("key", -INF), ("rotary", NAN), ("rotary", INF)])
def test_prefill_entry_that_is_seen(gpu_lib, new, seqs, heads, split, where, value):
    """Rows that see the entry as the formulas have them; the other rows, heads and requests the same bits."""
    import torch
    case = Prefill(new, seqs, heads=heads, seed=62)
    ws = gpu_lib.new_mla_workspace(1)
    if not split:
        ws = ws[:256].clone()
    f = lambda: gpu_lib.dsa_mla_prefill(*case.args(), entry_tokens=1, workspace=ws)  # noqa: E731
    want = [t.clone() for t in f()]
    t = case.entries[0] - 1 - new[0] // 2          # the first request's; about half of its rows see it
    if where == "key":
        case.kn[t, 0, 77] = value
    else:
        case.kr[t, 5] = value
    out, lse = f()
    for h in range(heads):
        o, l, _, seen = case.reference(0, h)
        got, got_l = out[:new[0], h], lse[:new[0], h]
        hit = seen > t if where == "rotary" or h == 0 else torch.zeros_like(seen, dtype=torch.bool)
        same_kind(got[hit], got_l[hit], o[hit], l[hit], f"head {h}")
        assert torch.equal(got[~hit], want[0][:new[0], h][~hit]) and torch.equal(got_l[~hit], want[1][:new[0], h][~hit])
        if hit.any() and value != value:
            assert torch.isnan(got_l[hit]).all()
    assert torch.equal(out[new[0]:], want[0][new[0]:]) and torch.equal(lse[new[0]:], want[1][new[0]:])
    assert torch.isnan(lse).any() or abs(value) == INF   # (an infinite score of the other sign has weight 0)
    assert gpu_lib.get_error(ws) == 0
