"""GPU tests of dsa_pages_update against a plain loop over the requests.  Whole numbers: all equal."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def plain(now, want, table, free, count, max_context, room):
    """The rule of include/dsa_indexer.h, request by request, on Python lists (all updated copies)."""
    pages = lambda n: -(-n // 256)  # noqa: E731
    now = [min(max(n, 0), max_context) for n in now]
    want = [min(max(n, 0), max_context) for n in want]
    table, free = [list(r) for r in table], list(free)
    good = lambda p: p if 0 <= p < len(free) else -1  # noqa: E731
    top = [good(p) for p in free[:count]]
    for b, (n, w) in enumerate(zip(now, want)):
        top += [good(p) for p in table[b][pages(w):pages(n)]]
    before = list(top)
    cu, slots, positions, lens, refused, asked = [0], [], [], [], False, 0
    for b, (n, w) in enumerate(zip(now, want)):
        if w > n:
            take, entries = range(pages(n), pages(w)), range(n // 4, -(-w // 4))
            asked += len(entries)
            refused = refused or len(take) > len(top) or asked > room
            if refused:
                w = n
            else:
                for i in take:
                    table[b][i] = top.pop()
                for e in entries:
                    page = good(table[b][e // 64])
                    slots.append(page * 64 + e % 64 if page >= 0 else -1)
                    positions.append(e)
        lens.append(w)
        cu.append(len(slots))
    for i in range(count, len(top)):
        free[i] = before[i]
    pad = [-1] * (room - len(slots))
    return table, free, lens, len(top), cu, slots + pad, positions + pad, refused


class State:
    def __init__(self, now, want, max_context, free, spare=0, seed=1):
        import torch
        rng = np.random.default_rng(seed)
        self.now, self.want, self.max_context, self.count = list(now), list(want), max_context, free
        used = [-(-min(max(n, 0), max_context) // 256) for n in now]
        self.pages = max(1, sum(used) + free + spare)
        ids = rng.permutation(self.pages).tolist()
        self.table = [[-1] * (max_context // 256) for _ in now]
        for row, n in zip(self.table, used):
            row[:n] = [ids.pop() for _ in range(n)]
        self.free = [ids.pop() for _ in range(free)]
        self.free += [-5] * (self.pages - free)
        ints = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        self.d = dict(seq_lens=ints(self.now), new_lens=ints(self.want), page_table=ints(self.table),
                      free_pages=ints(self.free), free_count=ints([free]))

    def args(self, room):
        d = self.d
        return d["seq_lens"], d["new_lens"], self.max_context, d["page_table"], d["free_pages"], d["free_count"], room

    def check(self, got, room):
        lens, count, cu, slots, positions = got
        want = plain(self.now, self.want, self.table, self.free, self.count, self.max_context, room)
        assert self.d["page_table"].tolist() == want[0]
        assert self.d["free_pages"].tolist() == want[1]
        assert lens.tolist() == want[2] and count.tolist() == [want[3]]
        assert cu.tolist() == want[4] and slots.tolist() == want[5] and positions.tolist() == want[6]
        return want


def run(lib, state, room, error=0, **kw):
    ws = lib.new_workspace(1, 256)
    got = lib.dsa_pages_update(*state.args(room), workspace=ws, **kw)
    assert lib.get_error(ws) == error
    assert not ws[:256].any()
    return state.check(got, room)


@pytest.mark.parametrize("now, want", [(0, 0), (0, 1), (1, 2), (3, 4), (4, 5), (255, 256), (256, 257), (0, 4096),
                                       (5, 4096), (4096, 0), (4096, 1), (300, 256), (257, 256), (300, 300)])
def test_pages_one_request(gpu_lib, now, want):
    run(gpu_lib, State([now], [want], 4096, 20, spare=2), 1100)


@pytest.mark.parametrize("batch", [1, 2, 31, 64, 257, 511, 512, 513, 1023, 1024])
@pytest.mark.parametrize("short", [False, True])
def test_pages_mixed(gpu_lib, batch, short):
    """Requests that end, shrink, stay, grow and arrive; with enough pages and slots, and with too few."""
    rng = np.random.default_rng(2 * batch + short)
    n = np.exp(rng.uniform(0, np.log(9000), batch)).astype(int)
    kind = rng.integers(6, size=batch)
    now = np.where(kind == 4, 0, n)
    want = np.select([kind == 0, kind == 1, kind == 2, kind == 3], [0, np.maximum(n - rng.integers(600, size=batch), 0), n,
                                                                   n + rng.integers(1, 5, size=batch)], n + 700 * (kind == 5))
    grow = want > now
    taken = int(np.maximum(-(-want // 256) - -(-now // 256), 0).sum())
    slots = int((-(-want // 4) - now // 4)[grow].sum())
    state = State(now.tolist(), want.tolist(), 10240, 0 if short else taken, spare=5, seed=batch)
    room = max(slots // 2, 1) if short and batch % 2 else slots + 3
    refused = plain(state.now, state.want, state.table, state.free, state.count, 10240, room)[-1]
    run(gpu_lib, state, room, error=gpu_lib.DEVERR_NO_PAGES if refused else 0)


def test_pages_large(gpu_lib):
    """Many slots and many returned pages: every CTA's part, odd room; 1M-token requests."""
    state = State([0, 1 << 20, 77, 1 << 19], [1 << 20, 0, 70000, (1 << 19) + 1], 1 << 20, 300, spare=9)
    run(gpu_lib, state, 262144 + 17482 + 5)
    run(gpu_lib, State([1 << 20] * 4, [0, 3, 1 << 19, 0], 1 << 20, 1), 1)


def test_pages_returned_pages_go_to_the_growing(gpu_lib):
    state = State([5000, 0, 3000], [100, 4000, 3001], 8192, 0)
    want = run(gpu_lib, state, 1024)
    assert not want[-1] and want[3] == 19 - 16


def test_pages_refusals_keep_the_rest(gpu_lib):
    """The first that does not fit and all later ones that grow stay; those that shrink do not."""
    state = State([100, 100, 100, 100, 5000], [600, 3000, 101, 102, 0], 8192, 0, spare=3)
    want = run(gpu_lib, state, 4096)
    assert want[2] == [600, 3000, 101, 102, 0]                       # 20 pages returned are enough
    state = State([100, 100, 100, 100, 600], [600, 3000, 101, 102, 0], 8192, 0, spare=3)
    want = run(gpu_lib, state, 4096, error=gpu_lib.DEVERR_NO_PAGES)
    assert want[2] == [600, 100, 100, 100, 0]
    state = State([0, 0, 0], [100, 100, 4], 256, 9)                  # slots for one and a half
    want = run(gpu_lib, state, 40, error=gpu_lib.DEVERR_NO_PAGES)
    assert want[2] == [100, 0, 0]


def test_pages_no_slots(gpu_lib):
    run(gpu_lib, State([700, 300], [0, 256], 1024, 3), 0)
    run(gpu_lib, State([700, 300], [701, 300], 1024, 3), 0, error=gpu_lib.DEVERR_NO_PAGES)


def test_pages_out_of_range(gpu_lib):
    """Lengths and counts out of range are held, bad ids are handed on as -1: nothing outside is touched."""
    import torch
    run(gpu_lib, State([-5, 5000, 300], [300, 100, 9000], 4096, 30), 2000, error=gpu_lib.DEVERR_SEQ_LEN_CLAMPED)
    state = State([700, 600], [1500, 0], 4096, 2, seed=3)
    state.table[0][2] = 999            # the page that holds its next entries, and a returned and a free one
    state.table[1][1] = -9
    state.free[1] = 1 << 30
    for k, v in (("page_table", state.table), ("free_pages", state.free)):
        state.d[k].copy_(torch.tensor(v, dtype=torch.int32))
    run(gpu_lib, state, 400, error=gpu_lib.DEVERR_BAD_PAGE)
    state = State([0, 700], [600, 0], 1024, 4)
    ws = gpu_lib.new_workspace(1, 256)
    for count in (-3, 1 << 30):        # results are not specified; nothing faults, the flag is set
        state.d["free_count"].fill_(count)
        gpu_lib.dsa_pages_update(*state.args(200), workspace=ws)
        assert gpu_lib.get_error(ws) & gpu_lib.DEVERR_BAD_RANGE


@pytest.mark.parametrize("batch, room", [(40, 300), (1000, 20000)])
def test_pages_in_place_over_steps(gpu_lib, batch, room):
    """A replayed graph that updates lengths and count in place, step after step, on one workspace."""
    import torch
    rng = np.random.default_rng(batch)
    now = rng.integers(1, 3000, size=batch).tolist()
    state = State(now, now, 8192, 60, spare=1)
    ws = gpu_lib.new_workspace(1, 256)
    d = state.d
    keep = dict(seq_lens_out=d["seq_lens"], free_count_out=d["free_count"])
    got = gpu_lib.dsa_pages_update(*state.args(room), workspace=ws, **keep)   # nothing changes
    state.check(got, room)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gpu_lib.dsa_pages_update(*state.args(room), workspace=ws, cu_slots=got[2], slots=got[3], positions=got[4], **keep)
    for step in range(8):
        state.now = d["seq_lens"].tolist()
        state.table, state.free, state.count = d["page_table"].tolist(), d["free_pages"].tolist(), int(d["free_count"])
        grow = rng.integers(0, 40, size=batch) * (rng.random(batch) < 0.7)
        state.want = np.where(rng.random(batch) < 0.1, 0, np.array(state.now) + grow).tolist()
        d["new_lens"].copy_(torch.tensor(state.want, dtype=torch.int32))
        graph.replay()
        state.check(got, room)
    assert gpu_lib.get_error(ws) & ~gpu_lib.DEVERR_NO_PAGES == 0
