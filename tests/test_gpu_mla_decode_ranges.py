"""GPU tests of dsa_mla_decode where a range ends with one block of a request behind another request's end: the
later one's partial must not be staged over the output of the earlier one while that is being stored."""
import pytest
from test_gpu_mla_decode import Case, run
from test_mla_dense_plan import plan, ranges_of  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def behind_and_whole(plan, seqs, next_n):  # noqa: F811
    """The requests that end just before a range's single last block of another, and those in one range."""
    import torch
    groups = torch.cuda.get_device_properties(0).multi_processor_count // next_n
    ranges, _ = ranges_of(plan, seqs, groups)
    behind = {r[-2][0] for r in ranges if len(r) > 1 and r[-1][2] - r[-1][1] == 1 and r[-1][3] > 1}
    return behind, {b for r in ranges for b, blo, bhi, nb, _ in r if blo == 0 and bhi == nb}


@pytest.mark.parametrize("next_n", [1, 2, 3, 4])
def test_decode_single_block_behind_a_whole_request(gpu_lib, plan, next_n):  # noqa: F811
    """Equal requests, and the same ones in reverse: those that are whole both times have the same bits."""
    import torch
    n = 301
    case = Case([2048] * n, 2048, next_n=next_n, seed=40 + next_n)
    behind, whole = behind_and_whole(plan, case.seqs, next_n)
    both = sorted(b for b in whole if n - 1 - b in whole)
    hit = sorted(behind & set(both))
    assert hit
    out, lse = [t.clone() for t in run(gpu_lib, case)]
    case.check(out, lse, rows=sorted(behind | set(range(0, n, 37))))
    for _ in range(10):
        again = run(gpu_lib, case)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    case.q, case.table = case.q.flip(0).contiguous(), case.table.flip(0).contiguous()
    back = run(gpu_lib, case)
    for b in both:
        assert torch.equal(out[b], back[0][n - 1 - b]) and torch.equal(lse[b], back[1][n - 1 - b]), b


@pytest.mark.parametrize("next_n", [1, 2, 4])
def test_decode_single_block_behind_a_partial(gpu_lib, plan, next_n):  # noqa: F811
    """64 requests of 8192 tokens: the output stored before is a partial's second half."""
    import torch
    case = Case([8192] * 64, 8192, next_n=next_n, seed=50 + next_n)
    behind, _ = behind_and_whole(plan, case.seqs, next_n)
    assert behind
    out, lse = [t.clone() for t in run(gpu_lib, case)]
    case.check(out, lse, rows=sorted(behind))
    for _ in range(10):
        again = run(gpu_lib, case)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
