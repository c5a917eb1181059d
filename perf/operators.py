"""Operators of the attention layer around the indexer, as a user's program calls them.

Three operators, each in its plain form (elementary torch operations in fp32) and,
with ``own`` set, through the package's entry points:

  norm     the residual's addition and the RMS norm of the hidden rows that feed the
           projections, with a bf16 output, an e4m3 output with fp32 scales, or both
  decode   latent attention, absorbed form: 1-4 query tokens per request over every
           live entry of the paged latent cache (64 heads, 576-wide entries)
  prefill  latent attention, expanded form: a ragged batch of prompts or prompt
           chunks, per-head keys (128 + 64 shared rotary dims) and values (128)

Lengths are part of a case (``lens_seed``), values come from the seed alone.
"""
import math
import random

import torch

own = False

EPS = 1e-6
HEADS, LATENT, VALUE, PAGE = 64, 576, 512, 64   # absorbed form: heads, entry width, value dims, entries per page
QK, NOPE, ROPE, DV = 192, 128, 64, 128          # expanded form: query/key width and its parts, value width
E4M3_MAX = 448.0


def listed():
    norm = dict(op="norm", stride=0, residual=True, bf16=True, group=0)
    dec = dict(op="decode", next_n=1, lens_seed=1)
    pre = dict(op="prefill", lens_seed=1)
    return [
        # one decoding request: the norm in front of the projections, for the bf16 indexer path and the 8-bit ones
        dict(norm, name="norm_one_token", rows=1, d=7168, group=128),
        # the dense decode batch
        dict(norm, name="norm_decode_b64", rows=64, d=7168),
        # the latent part of each token's 576-wide down-projection, a strided view, for a chunk of odd size
        dict(norm, name="norm_latent_4099", rows=4099, d=512, stride=576, residual=False),
        # a long prompt's hidden rows, 8 bits out for the projections
        dict(norm, name="norm_prefill_16k", rows=16384, d=7168, group=128, bf16=False),
        # one short request: 128 entries, latency only
        dict(dec, name="decode_b1_seq512", batch=1, max_context=8192, lens="full", longest=512),
        # one request at 1M context: the split over the cache's length does all the work
        dict(dec, name="decode_b1_ctx1m", batch=1, max_context=1 << 20, lens="full", longest=1 << 20),
        # mixed short requests with one draft token each (an empty request among them)
        dict(dec, name="decode_b16_ctx8k_mixed_q2", batch=16, next_n=2, max_context=8192, lens="mixed", longest=8192),
        # the dense batch: 64 requests at 128K context
        dict(dec, name="decode_b64_ctx128k", batch=64, max_context=131072, lens="full", longest=131072),
        # one short prompt on the compressed cache: 25 entries, latency only
        dict(pre, name="prefill_100", batch=1, heads=64, longest=100, past=0, entry_tokens=4, lens="full"),
        # a ragged batch of prompts of odd lengths (an empty one among them), one entry per token
        dict(pre, name="prefill_ragged_b7", batch=7, heads=32, longest=2047, past=0, entry_tokens=1, lens="mixed"),
        # one prompt of 8192 tokens
        dict(pre, name="prefill_8k", batch=1, heads=32, longest=8192, past=0, entry_tokens=1, lens="full"),
        # the last 1024-token chunk of a 128K prompt over the compressed cache
        dict(pre, name="prefill_chunk_128k", batch=1, heads=64, longest=1024, past=130048, entry_tokens=4,
             lens="full"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "decode", "prefill"])
    seed = rng.randrange(1 << 20)
    if op == "norm":
        d = rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 8, 1024), 64 * _log(rng, 1, 112)])
        rows = min(_log(rng, 1, 65536), (1 << 27) // (2 * d))
        group = rng.choice([0, 64, 128, -1])
        return dict(op=op, rows=rows, d=d, stride=rng.choice([0, 0, d + 64, d + 3]), residual=rng.random() < 0.6,
                    bf16=group == 0 or rng.random() < 0.5, group=group)
    if op == "decode":
        batch, next_n = _log(rng, 1, 96), rng.randrange(1, 5)
        longest = min(_log(rng, 1, 1 << 20), 64 * 131072 // (batch * next_n))
        ctx = -(-longest // 256) * 256 * rng.choice([1, 1, 2])
        return dict(op=op, batch=batch, next_n=next_n, max_context=ctx, lens=rng.choice(["full", "mixed"]),
                    longest=longest, lens_seed=seed)
    batch, heads = _log(rng, 1, 12), rng.choice([1, 2, 5, 8, 20, 32, 64, 128])
    entry_tokens = rng.choice([1, 4])
    longest = _log(rng, 1, 8192)
    past = rng.choice([0, _log(rng, 1, 65536)])
    entries = lambda: batch * heads * (-(-(past + longest) // entry_tokens))  # noqa: E731
    while entries() * longest > 1 << 31 or entries() > 1 << 21:
        batch, longest, past = -(-batch // 2), -(-longest * 2 // 3), past // 2
    return dict(op=op, batch=batch, heads=heads, longest=longest, past=past, entry_tokens=entry_tokens,
                lens=rng.choice(["full", "mixed"]), lens_seed=seed)


def _lengths(case):
    """Per request: new tokens (prefill) or the whole length (decode).  "mixed": spread over their
    logarithm up to the longest, which one request has; one more is empty where there are four or more."""
    n, most = case["batch"], case["longest"]
    if case["lens"] == "full":
        return [most] * n
    rng = random.Random(case["lens_seed"])
    lens = [_log(rng, 1, most) for _ in range(n)]
    lens[rng.randrange(n)] = most
    if n >= 4:
        lens[(lens.index(most) + 1) % n] = 0
    return lens


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, dtype=dtype, device="cuda", generator=gen)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        # hidden rows as they are: a spread of row magnitudes and a few large channels
        mag = torch.exp(normal(rows, 1, dtype=torch.float32))
        x = (normal(rows, case["stride"] or d, dtype=torch.float32) * mag)
        x[:, :: max(1, d // 7)] *= 8.0
        x = x.to(torch.bfloat16)[:, :d]
        return dict(case=case, x=x, residual=normal(rows, d) * 2 if case["residual"] else None,
                    weight=1 + 0.2 * normal(d))
    if case["op"] == "decode":
        batch, next_n, table_width = case["batch"], case["next_n"], case["max_context"] // 256
        lens = _lengths(case)
        pages = [_ceil(_ceil(n, 4), PAGE) for n in lens]
        total = max(1, sum(pages))
        perm = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
        table = torch.full((batch, table_width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, p in enumerate(pages):
            table[b, :p] = perm[at:at + p]
            at += p
        q = normal(*((batch, HEADS, LATENT) if next_n == 1 else (batch, next_n, HEADS, LATENT))) * 2
        return dict(case=case, q=q, kv=normal(total, PAGE, LATENT), table=table, seq_lens=ints(lens),
                    scale=QK ** -0.5, longest=max(lens))
    heads, e = case["heads"], case["entry_tokens"]
    new = _lengths(case)
    seq = [n + case["past"] if n else 0 for n in new]
    entries = [_ceil(n, e) for n in seq]
    cu = lambda v: [sum(v[:i]) for i in range(len(v) + 1)]  # noqa: E731
    kv = normal(max(1, sum(entries)), heads, NOPE + DV)      # one product makes both: keys and values are its views
    latent = normal(max(1, sum(entries)), LATENT)            # the rotary part is a view of the entry
    return dict(case=case, q=normal(sum(new), heads, QK) * 2, k_nope=kv[..., :NOPE], v=kv[..., NOPE:],
                k_rope=latent[:, VALUE:], cu_q=ints(cu(new)), cu_kv=ints(cu(entries)), seq_lens=ints(seq),
                scale=QK ** -0.5, most_q=max(new), most_kv=max(entries))


def run(state):
    case = state["case"]
    if own:
        return _own(state)
    if case["op"] == "norm":
        return _plain_norm(state)
    if case["op"] == "decode":
        return _plain_decode(state)
    return _plain_prefill(state)


def _own(s):
    from sparse_attention_paged_dsa_gb300 import binding as dsa
    case = s["case"]
    if case["op"] == "norm":
        if case["group"] == 0:
            return dsa.dsa_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"])
        return dsa.dsa_rmsnorm_fp8(s["x"], s["weight"], EPS, group=max(0, case["group"]), residual=s["residual"],
                                   with_bf16=case["bf16"])
    if case["op"] == "decode":
        if "workspace" not in s:  # kept by a serving loop
            s["workspace"] = dsa.new_mla_workspace(case["batch"], case["next_n"])
        return dsa.dsa_mla_decode(s["q"], s["kv"], s["table"], s["seq_lens"], case["max_context"], s["scale"],
                                  workspace=s["workspace"])
    if "workspace" not in s:
        s["workspace"] = dsa.new_mla_workspace(1)
    return dsa.dsa_mla_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_kv"], s["seq_lens"],
                               s["scale"], entry_tokens=case["entry_tokens"], workspace=s["workspace"])


def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    residual_out = None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        residual_out = h.to(torch.bfloat16)
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    out = y.to(torch.bfloat16) if case["bf16"] else None
    if case["group"] == 0:
        return out, residual_out
    rows, d = y.shape
    g = case["group"] if case["group"] > 0 else d
    padded = torch.nn.functional.pad(y, (0, _ceil(d, g) * g - d)).view(rows, -1, g)
    amax = padded.abs().amax(dim=2)
    scales = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    codes = (padded / scales[:, :, None]).reshape(rows, -1)[:, :d].to(torch.float8_e4m3fn)
    return codes, scales, out, residual_out


def _softmax_parts(scores, seen):
    """Weights, their sum and log-sum-exp over the last axis; where nothing is seen: zeros, 1 and -inf."""
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    return p, torch.where(total > 0, total, torch.ones_like(total)), lse


def _plain_decode(s):
    q, case = s["q"], s["case"]
    batch, next_n = case["batch"], case["next_n"]
    width = max(1, _ceil(s["longest"], 256))
    pages = s["table"][:, :width].clamp(min=0).long()
    kv = s["kv"][pages].view(batch, width * PAGE, LATENT).float()
    rows = q.reshape(batch, next_n * HEADS, LATENT).float()
    scores = torch.matmul(rows, kv.transpose(1, 2)).view(batch, next_n, HEADS, -1).mul_(s["scale"])
    back = torch.arange(next_n - 1, -1, -1, device="cuda")
    live = ((s["seq_lens"][:, None] - back).clamp(min=0) + 3) // 4                        # [batch, next_n]
    seen = torch.arange(width * PAGE, device="cuda") < live[:, :, None, None]
    p, total, lse = _softmax_parts(scores, seen)
    o = torch.matmul(p.view(batch, next_n * HEADS, -1), kv[:, :, :VALUE]).view(batch, next_n, HEADS, VALUE) / total
    return o.to(torch.bfloat16).view(*q.shape[:-1], VALUE), lse.view(q.shape[:-1])


def _plain_prefill(s):
    q, case = s["q"], s["case"]
    batch, heads, e = case["batch"], case["heads"], case["entry_tokens"]
    cu_q, cu_kv = s["cu_q"].long(), s["cu_kv"].long()
    i = torch.arange(max(1, s["most_q"]), device="cuda")
    t = torch.arange(max(1, s["most_kv"]), device="cuda")
    rows = (cu_q[:-1, None] + i).clamp(max=q.shape[0] - 1)                               # [batch, most_q]
    ents = (cu_kv[:-1, None] + t).clamp(max=s["v"].shape[0] - 1)                         # [batch, most_kv]
    key = torch.cat([s["k_nope"], s["k_rope"][:, None, :].expand(-1, heads, -1)], dim=2)
    qb = q[rows].float().transpose(1, 2)                                                 # [batch, heads, most_q, 192]
    kb = key[ents].float().permute(0, 2, 3, 1)
    scores = torch.matmul(qb, kb).mul_(s["scale"])
    new = cu_q[1:] - cu_q[:-1]
    length = s["seq_lens"].long()[:, None] - (new[:, None] - 1 - i)                      # tokens that row i sees
    seen = t < ((length.clamp(min=0) + e - 1) // e)[:, None, :, None]
    p, total, lse = _softmax_parts(scores, seen)
    o = torch.matmul(p, s["v"][ents].float().transpose(1, 2)) / total
    token = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(cu_q[1:], token, right=True)
    at = token - cu_q[b]
    return o[b, :, at].to(torch.bfloat16), lse[b, :, at]


def work(case):
    if case["op"] == "norm":
        rows, d, g = case["rows"], case["d"], case["group"]
        each = 2 + 4 * case["residual"] + 2 * case["bf16"] + (g != 0)
        scales = 0 if g == 0 else 4 * rows * (1 if g < 0 else _ceil(d, g))
        return dict(bytes=rows * d * each + scales + 2 * d, flops=rows * d * 6)
    if case["op"] == "decode":
        lens, next_n = _lengths(case), case["next_n"]
        entries = sum(_ceil(n, 4) for n in lens)
        pairs = sum(_ceil(max(0, n - j), 4) for n in lens for j in range(next_n))
        rows = case["batch"] * next_n * HEADS
        table = sum(4 * _ceil(n, 256) for n in lens)
        return dict(bytes=entries * LATENT * 2 + rows * (LATENT * 2 + VALUE * 2 + 4) + table + 4 * case["batch"],
                    flops=pairs * HEADS * (LATENT + VALUE) * 2)
    heads, e, past = case["heads"], case["entry_tokens"], case["past"]
    new = _lengths(case)
    entries = sum(_ceil(n + past, e) for n in new if n)
    pairs = 0
    for n in new:                        # sum over rows of ceil((past + 1 + i) / e)
        upto = lambda m: e * (m // e) * (m // e + 1) // 2 + (m % e) * (m // e + 1)  # noqa: E731
        pairs += upto(past + n) - upto(past) if n else 0
    return dict(bytes=sum(new) * heads * (QK * 2 + DV * 2 + 4) + entries * (heads * (NOPE + DV) + ROPE) * 2,
                flops=pairs * heads * (QK + DV) * 2)


# ------------------------------------------------------------------ 64 bits


def _to_e4m3(x):
    """Nearest e4m3 value (ties to even; 3 bits after the point, smallest exponent -6, at most 448)."""
    _, exponent = torch.frexp(x)
    step = torch.exp2((exponent - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        root = torch.sqrt(torch.sum(h ** 2, dim=1) / case["d"] + EPS)
        y = h / root[:, None] * s["weight"].double()
        kept = h if s["residual"] is not None else None
        if case["group"] == 0:
            return y, kept
        g = case["group"] if case["group"] > 0 else case["d"]
        scales, codes = [], []
        for piece in y.split(g, dim=1):
            most = piece.abs().max(dim=1, keepdim=True).values
            scale = torch.where(most > 0, most / E4M3_MAX, 1.0)
            scales.append(scale)
            codes.append(_to_e4m3(piece / scale))
        return torch.cat(codes, 1), torch.cat(scales, 1), y if case["bf16"] else None, kept
    if case["op"] == "decode":
        lens, next_n = _lengths(case), case["next_n"]
        q = s["q"].view(case["batch"], next_n, HEADS, LATENT)
        out = torch.zeros(case["batch"], next_n, HEADS, VALUE, dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], next_n, HEADS), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            whole = s["kv"][s["table"][b, :_ceil(_ceil(n, 4), PAGE)].long()].reshape(-1, LATENT)
            for j in range(next_n):
                live = _ceil(max(0, n - (next_n - 1 - j)), 4)
                if live:
                    kv = whole[:live].double()
                    x = s["scale"] * (kv @ q[b, j].double().T)             # [live, heads]
                    lse[b, j] = torch.logsumexp(x, dim=0)
                    out[b, j] = torch.exp(x - lse[b, j]).T @ kv[:, :VALUE]
        return out.view(*s["q"].shape[:-1], VALUE), lse.view(s["q"].shape[:-1])
    new, e, past = _lengths(case), case["entry_tokens"], case["past"]
    out = torch.zeros(sum(new), case["heads"], DV, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    at_q = at_kv = 0
    for n in new:
        entries = _ceil(n + past, e) if n else 0
        rotary = s["k_rope"][at_kv:at_kv + entries].double()
        upto = (torch.arange(n, device="cuda") + past + e) // e           # ceil((past + i + 1) / e)
        hidden = torch.arange(entries, device="cuda")[None, :] >= upto[:, None]
        for h in range(case["heads"] if n else 0):
            q = s["q"][at_q:at_q + n, h].double()
            x = q[:, :NOPE] @ s["k_nope"][at_kv:at_kv + entries, h].double().T + q[:, NOPE:] @ rotary.T
            x = (x * s["scale"]).masked_fill(hidden, -math.inf)
            lse[at_q:at_q + n, h] = torch.logsumexp(x, dim=1)
            out[at_q:at_q + n, h] = torch.softmax(x, dim=1) @ s["v"][at_kv:at_kv + entries, h].double()
        at_q, at_kv = at_q + n, at_kv + entries
    return out, lse
