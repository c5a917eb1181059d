"""GPU tests of the latent attentions where the running maximum is raised again and again over an accumulator that
holds something, at other blocks for other heads (rows), split and unsplit.

One of eight dims (of the rotary ones) is 1 in q, by head and row, and a multiple of 20 / scale in the keys, which
rises in steps within blocks: 20 nats are 28.9 log2 units, and the maximum is raised past 20.  The products of
these dims are exact, below 2048, and summed with ordinary ones: the sum is off by at most 8 steps of 2^-13, below
2^-13 after the scale; in log2 units a score is below 200 and its two roundings below 2^-16: a weight's relative
error stays under the 2^-12 that the bounds of the checks are made from.

What was summed before a raise counts for 2^-29 of it: half of the value dims are 2^28 times larger a step below the
top of one group, and 2^56 two steps below, so that there it counts as much (powers of 2: nothing is rounded), and
an accumulator scaled twice, or not at all, is seen."""
import pytest
from test_gpu_mla_decode import Case as Decode
from test_gpu_mla_decode import run as run_decode
from test_gpu_mla_prefill import Case as Prefill
from test_gpu_mla_prefill import run as run_prefill
from test_mla_dense_plan import plan, ranges_of  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

STEP, RAISE_LOG2, LOG2E = 20.0, 20.0, 1.4426950408889634


def raises(tops):
    """How often a running maximum that starts at the first block's top is raised: tops [..., blocks] in nats."""
    import torch
    m = tops[..., 0].clone()
    n = torch.zeros_like(m)
    for i in range(1, tops.shape[-1]):
        up = (tops[..., i] - m) * LOG2E > RAISE_LOG2
        n += up
        m = torch.where(up, tops[..., i], m)
    return n


@pytest.mark.parametrize("next_n, batch", [(1, 160), (2, 80), (4, 40)])
def test_decode_raises(gpu_lib, plan, next_n, batch):  # noqa: F811
    """Requests of 16 pages, whole or in parts of several, and of 4 pages (never cut)."""
    import torch
    seqs = [4096 - 4 * (b % 7) if b % 5 else 1024 for b in range(batch)]
    scale = 1.0 / 16
    case = Decode(seqs, 4096, next_n=next_n, seed=80 + next_n, scale=scale)
    group = (torch.arange(64, device="cuda") // 4) % 8    # of a head; heads 8 apart, which a thread shares, differ
    case.q[..., :256] = 0                                 # the value dims that grow take no part in the scores
    case.q[..., 512:520] = torch.nn.functional.one_hot(group, 8).to(torch.bfloat16)
    for b, s in enumerate(seqs):
        pages = -(-s // 256)
        t = torch.arange(pages * 64, device="cuda")[:, None]
        g = torch.arange(8, device="cuda")
        # rises by a step where the entry's place in its page passes 9 g, in every third page, 6 times at most
        level = ((t - 9 * g + 64 * 3) // (64 * 3) + (g + b) % 2).clamp(0, 6)
        rows = (case.table[b, :pages].long()[:, None] * 64 + torch.arange(64, device="cuda")).view(-1)
        flat = case.kv.view(-1, 576)
        flat[rows, 512:520] = (level * (STEP / scale)).to(torch.bfloat16)
        live = level[:case.live(b, next_n - 1), :1]
        flat[rows[:len(live)], :256] *= 2.0 ** (28 * (live.max() - live).clamp(max=2)).to(torch.bfloat16)
    ranges, _ = ranges_of(plan, seqs, torch.cuda.get_device_properties(0).multi_processor_count // next_n)
    total = most = 0
    for items in ranges:
        for b, blo, bhi, nb, _ in items:
            n = case.live(b, 0)
            t = torch.arange(n, device="cuda")
            kv = case.kv[case.table[b].long()[t // 64], t % 64].float()
            s = torch.full((64, nb * 64), -float("inf"), device="cuda")
            s[:, :n] = scale * (case.q[b, 0].float() @ kv.T)
            up = raises(s.view(64, nb, 64)[:, blo:bhi].amax(2))
            total, most = total + int(up.sum()), max(most, int(up.max()))
    assert total > 20 * batch and most >= 4, (total, most)
    out, lse = run_decode(gpu_lib, case)
    case.check(out, lse)
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("new, seqs, heads, split", [([600], [1400], 2, False), ([300, 129], [300, 900], 3, False),
                                                     ([1100], [1100], 1, False), ([1], [9999], 2, True),
                                                     ([130], [20000], 3, True), ([700], [9000], 3, True)])
def test_prefill_raises(gpu_lib, new, seqs, heads, split):
    """Tiles whose keys rise four times and fall back: any four tiles in a row, as the smallest part has, raise
    three or more of the five groups of rows and heads, one of them more than once."""
    import torch
    scale = 1.0 / 8
    case = Prefill(new, seqs, heads=heads, seed=90 + heads, scale=scale)
    for b in range(len(new)):
        q0, k0, n, m = case.cu_q_l[b], case.cu_kv_l[b], new[b], case.entries[b]
        group = (torch.arange(n, device="cuda")[:, None] // 8 + torch.arange(heads, device="cuda")) % 5
        case.q[q0:q0 + n, :, 128:133] = torch.nn.functional.one_hot(group, 5).to(torch.bfloat16)
        t, g = torch.arange(m, device="cuda")[:, None], torch.arange(5, device="cuda")
        level = ((t - 25 * g) // 128 + g) % 5             # rises within a tile for most groups
        case.kr[k0:k0 + m, :5] = (level * (STEP / scale)).to(torch.bfloat16)
        case.v[k0:k0 + m, :, :64] *= 2.0 ** (28 * (4 - level[:, :1, None]).clamp(max=2)).to(torch.bfloat16)
        tops = torch.stack([c.amax(0) for c in (level * STEP).float().split(128)], 1)   # [group, tile]
        for at in range(0, tops.shape[1] - 4, 3):
            up = raises(tops[:, at:at + 4])
            assert (up > 0).sum() >= 3 and up.max() >= 2
    out, lse = run_prefill(gpu_lib, case, split=split)
    case.check(out, lse)
    assert torch.isfinite(out.float()).all()
