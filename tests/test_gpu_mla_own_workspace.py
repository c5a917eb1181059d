"""GPU test of the latent attentions without a workspace: the one that a call makes for itself is of that call's
size, with nothing but its header cleared (all of it took longer than the kernel of short requests)."""
import pytest
from test_gpu_mla_decode import Case as Decode
from test_gpu_mla_prefill import Case as Prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_own_workspace_clears_its_header(gpu_lib, monkeypatch, kind):
    import torch
    if kind == "decode":
        case = Decode([100, 30], 512, seed=70)
        size, call = gpu_lib.mla_decode_workspace_size(2, 1), lambda **kw: gpu_lib.dsa_mla_decode(*case.args(), **kw)
    else:
        case = Prefill([20], [20], seed=71)
        size, call = gpu_lib.prefill_workspace_size(), lambda **kw: gpu_lib.dsa_mla_prefill(
            *case.args(), entry_tokens=1, **kw)
    want = [t.clone() for t in call(workspace=gpu_lib.new_mla_workspace(2))]
    made, space = [], gpu_lib._space
    monkeypatch.setattr(gpu_lib, "_space", lambda ws, device: made.append(ws) or space(ws, device))
    torch.cuda.empty_cache()
    torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")   # what the call's block holds before it
    got = call()
    assert len(made) == 1 and made[0].numel() == size
    assert not made[0][:256].any() and torch.all(made[0][-4096:] == 0x5A)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
