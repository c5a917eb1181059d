"""GPU tests of dsa_pages_update where a step drops tokens: what one call gives no slot for, two calls do."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

MAX = 4096


class Pages:
    def __init__(self, lib, batch, pages, seed):
        import torch
        g = torch.Generator().manual_seed(seed)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lib, self.lens, self.pages, self.room = lib, i32(batch), pages, batch * MAX // 4
        self.table = torch.full((batch, MAX // 256), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
        self.count = torch.full((1,), pages, dtype=torch.int32, device="cuda")
        self.ws = lib.new_workspace(batch, MAX)

    def go(self, want):
        """(entries, slots) of each request for these lengths."""
        import torch
        _, _, cu, slots, positions = self.lib.dsa_pages_update(
            self.lens, torch.tensor(want, dtype=torch.int32).cuda(), MAX, self.table, self.free, self.count, self.room,
            seq_lens_out=self.lens, free_count_out=self.count, workspace=self.ws)
        assert self.lens.tolist() == want and self.lib.get_error(self.ws) == 0
        cu, slots, positions, table = cu.tolist(), slots.tolist(), positions.tolist(), self.table.tolist()
        live = [p for row, n in zip(table, want) for p in row[: -(-n // 256)]]
        assert sorted(live + self.free[: int(self.count)].tolist()) == list(range(self.pages))
        out = []
        for b in range(len(want)):
            mine = list(zip(positions[cu[b]:cu[b + 1]], slots[cu[b]:cu[b + 1]]))
            assert all(s == table[b][e // 64] * 64 + e % 64 for e, s in mine)
            out.append([e for e, _ in mine])
        return out


@pytest.mark.parametrize("batch, seed", [(1, 0), (7, 1), (130, 2), (1024, 3)])
def test_two_calls_for_a_step_that_drops_tokens(gpu_lib, batch, seed):
    """Kept lengths of every remainder, on a page's border too; some requests only roll back, some also grow."""
    rng = np.random.default_rng(seed)
    have = rng.integers(1, 3000, batch)
    have[:: 3] = np.minimum(have[:: 3] // 256 * 256 + rng.integers(1, 9, len(have[:: 3])), 3000)
    state = Pages(gpu_lib, batch, 16 * batch + 4, seed)
    state.go(have.tolist())
    for _ in range(3):
        kept = np.maximum(have - rng.integers(0, 9, batch), 0)
        new = np.where(rng.random(batch) < 0.5, kept, np.minimum(kept + rng.integers(0, 600, batch), MAX - 8))
        assert not any(state.go(kept.tolist())) or (kept == have).all()       # one call that shrinks: no slots
        state.go((kept // 4 * 4).tolist())
        entries = state.go(new.tolist())
        assert entries == [list(range(k // 4, -(-n // 4))) for k, n in zip(kept.tolist(), new.tolist())]
        have = new
