"""Operators around the paged caches, as a serving program calls them.

Three operators, each in its plain form (elementary torch operations) and, with
``own`` set, through the package's entry points:

  pages   the requests' page-table rows, their lengths, the list of free pages and the
          slots of the entries to be written, from the lengths of now and of the next step
  append  new entries into the paged caches at their slots: RMS norm and rotation of the
          latent entries, norm and 8-bit quantisation of the index keys
  tree    latent attention, absorbed form, for a tree of drafted tokens: every live entry
          of the paged cache, and the drafted tokens that the tree's mask shows

Lengths are part of a case (``lens_seed``), values come from the seed alone.
"""
import math
import random

import torch

own = False

EPS = 1e-6
HEADS, LATENT, VALUE, ROPE, KEY = 64, 576, 512, 64, 64   # entry: 512 value dims and 64 rotary ones; index keys of 64
PAGE, TOKENS = 64, 4                                     # entries per page, tokens per entry
PAGE_TOKENS = PAGE * TOKENS
E4M3_MAX = 448.0


def listed():
    pages = dict(op="pages", lens_seed=1, short=False)
    app = dict(op="append", latent=True, norm=True, rope=True, keys="fp8", wide=False)
    tree = dict(op="tree", lens_seed=1, ragged=False)
    return [
        # one decode step of 64 long requests, each with one to four tokens more: latency only
        dict(pages, name="pages_step_b64", batch=64, kind="step", longest=131072, max_context=131072),
        # a busy server between two steps, with too few pages: requests end, roll back drafted tokens, grow, arrive
        dict(pages, name="pages_churn_b257_short", batch=257, kind="churn", longest=20011, max_context=32768,
             short=True),
        # admission of 1024 prompts at once
        dict(pages, name="pages_admit_b1024", batch=1024, kind="admit", longest=8192, max_context=8192),
        # one entry of one decoding request: latency only
        dict(app, name="append_one", rows=1),
        # the step of 64 requests into caches whose rows are already normed: bf16 index keys, nothing computed
        dict(app, name="append_b64_plain", rows=64, norm=False, rope=False, keys="bf16"),
        # a chunk of odd size, latents and index keys as views of one wide product
        dict(app, name="append_4099_wide", rows=4099, wide=True),
        # the entries of a 1M-token prompt on the compressed cache
        dict(app, name="append_262144", rows=262144),
        # eight drafted tokens of one short request: latency only
        dict(tree, name="tree_b1_t8_seq512", batch=1, tokens=8, lens="full", longest=512),
        # a batch of short requests of mixed lengths with trees of different sizes (an empty request among them)
        dict(tree, name="tree_b13_t27_8k_ragged", batch=13, tokens=27, lens="mixed", longest=8192, ragged=True),
        # one long request, sixteen drafted tokens: the split over the cache's length does all the work
        dict(tree, name="tree_b1_t16_ctx128k", batch=1, tokens=16, lens="full", longest=131072),
        # many long requests with a chain of two: the cache's bytes count
        dict(tree, name="tree_b64_t2_ctx64k", batch=64, tokens=2, lens="full", longest=65536),
        # a batch of long requests, 32 drafted tokens each: the products count
        dict(tree, name="tree_b16_t32_ctx128k", batch=16, tokens=32, lens="full", longest=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _ceil(a, b):
    return -(-a // b)


def draw(rng):
    op = rng.choice(["pages", "append", "tree"])
    seed = rng.randrange(1 << 20)
    if op == "pages":
        batch = _log(rng, 1, 1024)
        longest = min(_log(rng, 1, 1 << 20), (1 << 23) // batch)
        return dict(op=op, batch=batch, kind=rng.choice(["step", "churn", "admit"]), longest=longest,
                    max_context=_ceil(longest + 4, PAGE_TOKENS) * PAGE_TOKENS * rng.choice([1, 1, 2]),
                    short=rng.random() < 0.3, lens_seed=seed)
    if op == "append":
        latent = rng.random() < 0.8
        keys = rng.choice(["fp8", "fp8", "bf16", "none"]) if latent else rng.choice(["fp8", "bf16"])
        return dict(op=op, rows=_log(rng, 1, 262144), latent=latent, norm=rng.random() < 0.7,
                    rope=latent and rng.random() < 0.7, keys=keys, wide=latent and rng.random() < 0.4)
    batch, tokens = _log(rng, 1, 96), _log(rng, 1, 64)
    longest = min(_log(rng, 1, 1 << 20), 16 * 32 * 131072 // (batch * max(2, tokens)))
    return dict(op=op, batch=batch, tokens=tokens, lens=rng.choice(["full", "mixed"]), longest=longest,
                ragged=rng.random() < 0.5, lens_seed=seed)


# ------------------------------------------------------------------ lengths


def _lengths(case):
    """Tokens per request.  "mixed": spread over their logarithm up to the longest, which one request
    has; one more is empty where there are four or more."""
    n, most = case["batch"], case["longest"]
    if case["lens"] == "full":
        return [most] * n
    rng = random.Random(case["lens_seed"])
    lens = [_log(rng, 1, most) for _ in range(n)]
    lens[rng.randrange(n)] = most
    if n >= 4:
        lens[(lens.index(most) + 1) % n] = 0
    return lens


def _counts(case):
    """Drafted tokens per request."""
    if not case["ragged"]:
        return [case["tokens"]] * case["batch"]
    rng = random.Random(case["lens_seed"] + 1)
    return [rng.randint(0 if case["batch"] > 2 else 1, case["tokens"]) for _ in range(case["batch"])]


def _changes(case):
    """(lengths now, lengths wanted, free pages, room for slots) of a page step."""
    rng = random.Random(case["lens_seed"])
    now, want, most = [], [], case["longest"]
    for _ in range(case["batch"]):
        n = _log(rng, 1, most)
        kind = case["kind"] if case["kind"] != "churn" else rng.choices(
            ["end", "back", "step", "admit", "same"], [20, 15, 40, 15, 10])[0]
        now.append(0 if kind == "admit" else n)
        want.append(dict(step=min(n + rng.randint(1, 4), case["max_context"]), end=0, same=n, admit=n,
                         back=max(0, n - rng.randint(1, 300)))[kind])
    pages = lambda n: _ceil(n, PAGE_TOKENS)  # noqa: E731
    taken = sum(max(0, pages(w) - pages(n)) for n, w in zip(now, want))
    freed = sum(max(0, pages(n) - pages(w)) for n, w in zip(now, want))
    slots = sum(_ceil(w, TOKENS) - n // TOKENS for n, w in zip(now, want) if w > n)
    free = max(0, (taken * 3) // 4 - freed) if case["short"] else taken + case["batch"] // 3
    return now, want, free, slots + slots // 16 + 1


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, dtype=dtype, device="cuda", generator=gen)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device="cuda")

    if case["op"] == "pages":
        now, want, free, room = _changes(case)
        width = case["max_context"] // PAGE_TOKENS
        used = [_ceil(n, PAGE_TOKENS) for n in now]
        total = sum(used) + free + case["batch"]                # some pages belong to others
        perm = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
        live = torch.arange(width, device="cuda") < ints(used)[:, None]
        table[live] = perm[:sum(used)]
        stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        stack[:free] = perm[sum(used):sum(used) + free]
        return dict(case=case, seq_lens=ints(now), new_lens=ints(want), table=table, free_pages=stack,
                    free_count=ints([free]), room=room)
    if case["op"] == "append":
        rows = case["rows"]
        pages = _ceil(rows, PAGE) + max(1, rows // (4 * PAGE))
        slots = torch.randperm(pages * PAGE, device="cuda", generator=gen)[:rows]
        slots[torch.rand(rows, device="cuda", generator=gen) < 0.02] = -1   # places that no entry has come to yet
        wide = normal(rows, LATENT + KEY + 64) if case["wide"] else None
        s = dict(case=case, slots=slots, latent=None, weight=None, cos_sin=None, positions=None, kv=None, keys=None,
                 key_weight=None, pool=None, codes=None, scales=None)
        if case["latent"]:
            s["latent"] = wide[:, :LATENT] if case["wide"] else normal(rows, LATENT)
            s["kv"] = normal(pages, PAGE, LATENT)
            if case["norm"]:
                s["weight"] = 1 + 0.2 * normal(VALUE)
            if case["rope"]:
                far = 1 << 18
                angles = torch.outer(torch.arange(far, device="cuda", dtype=torch.float64) * TOKENS,
                                     10000.0 ** (-torch.arange(ROPE // 2, device="cuda", dtype=torch.float64) / 32))
                s["cos_sin"] = torch.cat([torch.cos(angles), torch.sin(angles)], 1).float()
                s["positions"] = torch.randint(far, (rows,), device="cuda", generator=gen, dtype=torch.int32)
        if case["keys"] != "none":
            s["keys"] = wide[:, LATENT:LATENT + KEY] if case["wide"] else normal(rows, KEY)
            if case["norm"]:
                s["key_weight"] = 1 + 0.2 * normal(KEY)
            if case["keys"] == "bf16":
                s["pool"] = normal(pages, PAGE, KEY)
            else:
                s["codes"] = normal(pages, PAGE, KEY, dtype=torch.float32).to(torch.float8_e4m3fn)
                s["scales"] = torch.exp(normal(pages, PAGE, dtype=torch.float32))
        return s
    batch, tokens = case["batch"], case["tokens"]
    lens, counts = _lengths(case), _counts(case)
    width = max(1, _ceil(max(lens), PAGE_TOKENS))
    used = [_ceil(n, PAGE_TOKENS) for n in lens]
    total = max(1, sum(used))
    perm = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda") < ints(used)[:, None]] = perm[:sum(used)]
    rng = random.Random(seed)
    masks = []
    for _ in range(batch):
        seen = []                                              # each token: its parent's ancestors and itself
        for j in range(tokens):
            parent = rng.randint(max(-1, j - 4), j - 1)
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        masks.append([m - (1 << 64) if m >> 63 else m for m in seen])
    return dict(case=case, q=normal(batch, tokens, HEADS, LATENT) * 2, kv=normal(total, PAGE, LATENT), table=table,
                seq_lens=ints(lens), draft=normal(batch, tokens, LATENT), mask=ints(masks, torch.int64),
                counts=ints(counts) if case["ragged"] else None, scale=192 ** -0.5,
                out=torch.zeros(batch, tokens, HEADS, VALUE, dtype=torch.bfloat16, device="cuda"),
                lse=torch.zeros(batch, tokens, HEADS, device="cuda"), max_context=width * PAGE_TOKENS)


def run(state):
    if own:
        return _own(state)
    return {"pages": _plain_pages, "append": _plain_append, "tree": _plain_tree}[state["case"]["op"]](state)


def _own(s):
    from sparse_attention_paged_dsa_gb300 import binding as dsa
    case = s["case"]
    if case["op"] == "pages":
        if "workspace" not in s:  # kept by a serving loop
            s["workspace"] = dsa.new_workspace(case["batch"], case["max_context"])
        lens, count, cu, slots, positions = dsa.dsa_pages_update(
            s["seq_lens"], s["new_lens"], case["max_context"], s["table"], s["free_pages"], s["free_count"], s["room"],
            workspace=s["workspace"])
        return s["table"], s["free_pages"], lens, count, cu, slots, positions
    if case["op"] == "append":
        if "workspace" not in s:
            s["workspace"] = dsa.new_workspace(1, PAGE_TOKENS)
        dsa.dsa_cache_append(s["slots"], latent=s["latent"], latent_weight=s["weight"], cos_sin=s["cos_sin"],
                             positions=s["positions"], kv_cache=s["kv"], index_keys=s["keys"],
                             index_weight=s["key_weight"], key_pool=s["pool"], key_codes=s["codes"],
                             key_scales=s["scales"], eps=EPS, workspace=s["workspace"])
        return s["kv"], s["pool"], s["codes"], s["scales"]
    if "workspace" not in s:
        s["workspace"] = dsa.new_tree_workspace(case["batch"], case["tokens"])
    return dsa.dsa_mla_tree_decode(s["q"], s["kv"], s["table"], s["seq_lens"], s["max_context"], s["draft"], s["mask"],
                                   s["scale"], token_counts=s["counts"], out=s["out"], lse=s["lse"],
                                   workspace=s["workspace"])


# ------------------------------------------------------------------ plain forms


def _plain_pages(s):
    old, want, count, room = s["seq_lens"].long(), s["new_lens"].long(), s["free_count"].long(), s["room"]
    table, stack = s["table"], s["free_pages"]
    have, need = (old + 255) // 256, (want + 255) // 256
    grow = want > old
    take, give = (need - have).clamp(min=0), (have - need).clamp(min=0)
    n = torch.where(grow, (want + 3) // 4 - old // 4, torch.zeros_like(old))
    given = torch.cumsum(give, 0)
    avail = count + given[-1:]
    served = ~grow | ((torch.cumsum(take, 0) <= avail) & (torch.cumsum(n, 0) <= room))
    take, n = take * served, n * served
    lens = torch.where(served, want, old)
    # the free pages with the returned ones on top
    at = torch.arange(stack.shape[0], device="cuda")
    k = at - count
    b = torch.searchsorted(given, k.clamp(min=0), right=True).clamp(max=len(old) - 1)
    place = (need[b] + k - (given[b] - give[b])).clamp(0, table.shape[1] - 1)
    top = torch.where((k >= 0) & (at < avail), table[b, place], stack)
    taken = torch.cumsum(take, 0)
    left = avail - taken[-1:]
    # pages from the top, request by request
    w = torch.arange(table.shape[1], device="cuda")
    kth = (taken - take - have)[:, None] + w
    fresh = (w >= have[:, None]) & (w < need[:, None]) & (take > 0)[:, None]
    table.copy_(torch.where(fresh, top[(avail - 1 - kth).clamp(0, stack.shape[0] - 1)], table))
    stack.copy_(torch.where(at < left, top, stack))
    cu = torch.cat([torch.zeros_like(count), torch.cumsum(n, 0)])
    i = torch.arange(room, device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=len(old) - 1)
    entry = old[b] // 4 + i - cu[b]
    real = i < cu[-1]
    page = table[b, (entry // PAGE).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(real, page * PAGE + entry % PAGE, torch.full_like(i, -1))
    positions = torch.where(real, entry, torch.full_like(i, -1))
    return table, stack, lens.int(), left.int(), cu.int(), slots, positions.int()


def _norm(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * weight.float()


def _plain_append(s):
    # the row that comes to each slot, or -1 (rows without a slot meet in front of the first one)
    places = next(s[c].shape[0] for c in ("kv", "pool", "codes") if s[c] is not None) * PAGE
    row = torch.full((places + 1,), -1, dtype=torch.int64, device="cuda")
    row[s["slots"] + 1] = torch.arange(len(s["slots"]), device="cuda")
    row = row[1:]
    come = row >= 0

    def put(cache, values):
        flat = cache.view(places, -1)
        flat.copy_(torch.where(come[:, None], values.view(len(s["slots"]), -1)[row.clamp(min=0)], flat))

    if s["latent"] is not None:
        x = s["latent"].float()
        rotary = x[:, VALUE:]
        if s["cos_sin"] is not None:
            c, d = s["cos_sin"][s["positions"].long()].chunk(2, dim=1)
            a, b = rotary[:, 0::2], rotary[:, 1::2]
            rotary = torch.stack([a * c - b * d, a * d + b * c], dim=2).flatten(1)
        entry = torch.cat([_norm(x[:, :VALUE], s["weight"]), rotary], dim=1).to(torch.bfloat16)
        put(s["kv"], entry)
    if s["keys"] is not None:
        y = _norm(s["keys"].float(), s["key_weight"])
        if s["pool"] is not None:
            put(s["pool"], y.to(torch.bfloat16))
        else:
            most = y.abs().amax(dim=1)
            scale = torch.where(most > 0, most / E4M3_MAX, torch.ones_like(most))
            codes = (y / scale[:, None]).to(torch.float8_e4m3fn)
            put(s["codes"].view(torch.uint8), codes.view(torch.uint8))
            put(s["scales"], scale)
    return s["kv"], s["pool"], s["codes"], s["scales"]


def _plain_tree(s):
    case, q = s["case"], s["q"]
    batch, tokens = case["batch"], case["tokens"]
    width = s["table"].shape[1]
    kv = s["kv"][s["table"].clamp(min=0).long()].view(batch, width * PAGE, LATENT)
    kv = torch.cat([kv, s["draft"]], dim=1).float()
    scores = torch.matmul(q.view(batch, tokens * HEADS, LATENT).float(), kv.transpose(1, 2)).mul_(s["scale"])
    scores = scores.view(batch, tokens, HEADS, -1)
    live = torch.arange(width * PAGE, device="cuda") < ((s["seq_lens"].long() + 3) // 4)[:, None]
    drafted = (s["mask"][:, :, None] >> torch.arange(tokens, device="cuda")) & 1 != 0
    written = torch.ones(batch, tokens, dtype=torch.bool, device="cuda")
    if s["counts"] is not None:
        written = torch.arange(tokens, device="cuda") < s["counts"][:, None]
        drafted = drafted & written[:, None, :]
    seen = torch.cat([live[:, None, :].expand(-1, tokens, -1), drafted], dim=2)[:, :, None, :]
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    o = torch.matmul(p.view(batch, tokens * HEADS, -1), kv[:, :, :VALUE]).view(batch, tokens, HEADS, VALUE)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(torch.where(written[:, :, None, None], o.to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(written[:, :, None], lse, s["lse"]))
    return s["out"], s["lse"]


# ------------------------------------------------------------------ work


def work(case):
    if case["op"] == "pages":
        now, want, free, room = _changes(case)
        pages = lambda n: _ceil(n, PAGE_TOKENS)  # noqa: E731
        moved = sum(abs(pages(w) - pages(n)) for n, w in zip(now, want))
        return dict(bytes=case["batch"] * 16 + moved * 8 + room * 12, flops=room)
    if case["op"] == "append":
        rows, latent, keys = case["rows"], case["latent"], case["keys"]
        each = 8 + latent * 2 * LATENT * 2 + (KEY * 2 if keys != "none" else 0)
        each += {"none": 0, "bf16": KEY * 2, "fp8": KEY + 4}[keys] + case["rope"] * (4 + ROPE * 4)
        return dict(bytes=rows * each, flops=rows * (latent * VALUE * 4 * case["norm"] + KEY * 6))
    lens, counts = _lengths(case), _counts(case)
    entries = sum(_ceil(n, TOKENS) for n, c in zip(lens, counts) if c)
    pairs = sum(c * _ceil(n, TOKENS) + c * (c + 1) // 2 for n, c in zip(lens, counts))
    rows = sum(counts) * HEADS
    return dict(bytes=(entries + sum(counts)) * LATENT * 2 + rows * (LATENT * 2 + VALUE * 2 + 4) + 8 * sum(counts),
                flops=pairs * HEADS * (LATENT + VALUE) * 2)


# ------------------------------------------------------------------ 64 bits


def _to_e4m3(x):
    """Nearest e4m3 value (ties to even; 3 bits after the point, smallest exponent -6, at most 448)."""
    _, exponent = torch.frexp(x)
    step = torch.exp2((exponent - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    if case["op"] == "pages":
        s = prepare(case, seed)
        now, want, free, room = _changes(case)
        table, stack = s["table"].tolist(), s["free_pages"].tolist()
        top = stack[:free]
        for b, (n, w) in enumerate(zip(now, want)):
            if w < n:
                top += table[b][_ceil(w, PAGE_TOKENS):_ceil(n, PAGE_TOKENS)]
        cu, slots, positions, lens, full, asked = [0], [], [], [], False, 0
        for b, (n, w) in enumerate(zip(now, want)):
            if w > n:
                pages = range(_ceil(n, PAGE_TOKENS), _ceil(w, PAGE_TOKENS))
                entries = range(n // TOKENS, _ceil(w, TOKENS))
                full = full or len(pages) > len(top) or asked + len(entries) > room   # and nobody after it
                asked += len(entries)
                if full:
                    w = n
                else:
                    for page in pages:
                        table[b][page] = top.pop()
                    slots += [table[b][e // PAGE] * PAGE + e % PAGE for e in entries]
                    positions += entries
            lens.append(w)
            cu.append(len(slots))
        stack[:len(top)] = top
        pad = [-1] * (room - len(slots))
        values = (table, stack, lens, [len(top)], cu, slots + pad, positions + pad)
        return tuple(torch.tensor(v, dtype=torch.int64, device="cuda") for v in values)
    if case["op"] == "append":
        s = prepare(case, seed)
        rows = torch.nonzero(s["slots"] >= 0)[:, 0]
        to = s["slots"][rows]

        def normed(x, weight):
            x = x.double()
            if weight is not None:
                x = x / torch.sqrt(torch.sum(x ** 2, dim=1, keepdim=True) / x.shape[1] + EPS) * weight.double()
            return x

        kv = pool = codes = scales = None
        if case["latent"]:
            x = s["latent"][rows]
            kv = s["kv"].double()
            flat = kv.view(-1, LATENT)
            flat[to, :VALUE] = normed(x[:, :VALUE], s["weight"])
            z = torch.view_as_complex(x[:, VALUE:].double().reshape(-1, ROPE // 2, 2))
            if case["rope"]:
                table = s["cos_sin"].double()[s["positions"].long()[rows]]
                z = z * torch.complex(table[:, :ROPE // 2], table[:, ROPE // 2:])
            flat[to, VALUE:] = torch.view_as_real(z).reshape(-1, ROPE)
        if case["keys"] != "none":
            y = normed(s["keys"][rows], s["key_weight"])
            if case["keys"] == "bf16":
                pool = s["pool"].double()
                pool.view(-1, KEY)[to] = y
            else:
                codes, scales = s["codes"].to(torch.float32).double(), s["scales"].double()
                most = torch.max(torch.abs(y), dim=1, keepdim=True).values
                scale = torch.where(most > 0, most / E4M3_MAX, 1.0)
                codes.view(-1, KEY)[to] = _to_e4m3(y / scale)
                scales.view(-1)[to] = scale[:, 0]
        return kv, pool, codes, scales
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    out, lse = s["out"].double(), s["lse"].double()
    masks = s["mask"].tolist()
    for b, (n, count) in enumerate(zip(_lengths(case), _counts(case))):
        pages = s["table"][b, :_ceil(n, PAGE_TOKENS)].long()
        cache = s["kv"][pages].reshape(-1, LATENT)[:_ceil(n, TOKENS)].double()
        for j in range(count):
            seen = [i for i in range(count) if masks[b][j] >> i & 1]
            kv = torch.cat([cache, s["draft"][b, seen].double()])
            if not len(kv):
                out[b, j], lse[b, j] = 0, -math.inf
                continue
            x = s["scale"] * (kv @ s["q"][b, j].double().T)                # [entries, heads]
            lse[b, j] = torch.logsumexp(x, dim=0)
            out[b, j] = torch.exp(x - lse[b, j]).T @ kv[:, :VALUE]
    return out, lse
