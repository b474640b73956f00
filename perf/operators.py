"""The cases that the pool operators are measured by: norms and rotary positions, sliding-window attention, shared prefixes.

Three operators of one serving step over the paged KV pool (64 query heads, 8 KV heads, 128 dims, 64-token chunks):

* ``norm_rope``: the norms of queries and keys for each head and the rotary positions, from one row of the fused
  projection, with K and V written dense or into the pool's chunks;
* ``window``: attention of each query over the last ``window`` tokens and the first ``sinks`` ones;
* ``prefix``: one decode step of a batch whose groups share a long prefix, read once for the whole group.

``run`` computes them in elementary torch operations in 32 bits (angles in 64), or, with ``own``, by the calls that a
user makes of the library.
"""
import math
import random

import torch

own = False

HEADS, KV, DIM, CHUNK = 64, 8, 128, 64
GROUP = HEADS // KV
WIDTH = (HEADS + 2 * KV) * DIM
EPS = 1e-6


def listed():
    return [
        # One decoded token of one sequence at a far position: what counts is the latency of the call.
        {"name": "rope_token", "op": "norm_rope", "tokens": 1, "layout": "half", "rot": 128, "norm": True, "pool": False,
         "pad": 0, "factor": 1.0, "far": 1000000},
        # One decode step of a batch, part of each head rotated in interleaved pairs, frequencies stretched by 4.
        {"name": "rope_batch_pool", "op": "norm_rope", "tokens": 32, "layout": "interleaved", "rot": 64, "norm": True,
         "pool": True, "pad": 0, "factor": 4.0, "far": 262144},
        # A long prompt's projection into the pool, from rows of a wider buffer.
        {"name": "rope_prompt_pool", "op": "norm_rope", "tokens": 8191, "layout": "half", "rot": 128, "norm": True,
         "pool": True, "pad": 64, "factor": 1.0, "far": 8191},
        # One decoded token of one long sequence.
        {"name": "window_token", "op": "window", "batch": 1, "queries": 1, "longest": 524287, "window": 4096, "sinks": 4,
         "ragged": 1},
        # One decode step of a ragged batch, its shortest sequences shorter than the window.
        {"name": "window_decode", "op": "window", "batch": 64, "queries": 1, "longest": 131072, "window": 1024, "sinks": 4,
         "ragged": 2},
        # A prompt from its first token.
        {"name": "window_prompt", "op": "window", "batch": 1, "queries": 4096, "longest": 4096, "window": 1024, "sinks": 4,
         "ragged": 3},
        # Pieces of prompts and single tokens in one batch, behind what was cached before.
        {"name": "window_pieces", "op": "window", "batch": 6, "queries": 1000, "longest": 16384, "window": 4096, "sinks": 64,
         "ragged": 4},
        # Four samples drawn for one short prompt.
        {"name": "prefix_samples", "op": "prefix", "groups": 1, "batch": 4, "prefix": 1000, "suffix": 64, "ragged": 5},
        # A batch of questions on one long document.
        {"name": "prefix_document", "op": "prefix", "groups": 1, "batch": 32, "prefix": 32768, "suffix": 1024, "ragged": 6},
        # A large batch under several instructions of different lengths.
        {"name": "prefix_groups", "op": "prefix", "groups": 5, "batch": 128, "prefix": 16384, "suffix": 512, "ragged": 7},
    ]


def _log_int(rng, low, high):
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["norm_rope", "window", "window", "prefix"])
    if op == "norm_rope":
        tokens = _log_int(rng, 1, 8191)
        return {"op": op, "tokens": tokens, "layout": rng.choice(["half", "interleaved"]), "rot": 8 * rng.randint(2, 16),
                "norm": rng.random() < 0.8, "pool": rng.random() < 0.7, "pad": 8 * rng.randint(0, 16),
                "factor": rng.choice([1.0, 4.0, 16.0]), "far": _log_int(rng, tokens, 1000000)}
    if op == "window":
        ragged, window, sinks = rng.randrange(1 << 20), _log_int(rng, 32, 4096), rng.randint(0, 100)
        if rng.random() < 0.5:
            return {"op": op, "batch": _log_int(rng, 1, 64), "queries": 1, "longest": _log_int(rng, 64, 131072),
                    "window": window, "sinks": sinks, "ragged": ragged}
        batch, queries = _log_int(rng, 1, 6), _log_int(rng, 2, 4096)
        window = min(window, 4200000 // (batch * queries) - sinks)
        return {"op": op, "batch": batch, "queries": queries, "longest": _log_int(rng, queries, 16384), "window": window,
                "sinks": sinks, "ragged": ragged}
    batch = _log_int(rng, 1, 128)
    return {"op": op, "groups": min(batch, rng.randint(1, 5)), "batch": batch, "prefix": _log_int(rng, 32, 16384),
            "suffix": _log_int(rng, 1, 512), "ragged": rng.randrange(1 << 20)}


# ---------------------------------------------------------------- sizes that a case fixes
def _window_lengths(case):
    """Queries and cached tokens of each sequence: the first has the case's own, the others fewer."""
    r = random.Random(case["ragged"])
    q = [case["queries"]] + [_log_int(r, 1, case["queries"]) for _ in range(case["batch"] - 1)]
    n = [case["longest"]] + [r.randint(x, max(x, case["longest"])) for x in q[1:]]
    return q, n


def _prefix_lengths(case):
    """Sequences of each group, the groups' prefix lengths and the sequences' own lengths."""
    r = random.Random(case["ragged"])
    cuts = sorted(r.sample(range(1, case["batch"]), case["groups"] - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [case["batch"]])]
    prefix = [case["prefix"]] + [_log_int(r, max(1, case["prefix"] // 16), case["prefix"]) for _ in sizes[1:]]
    return sizes, prefix, [case["suffix"]] + [r.randint(0, case["suffix"]) for _ in range(case["batch"] - 1)]


def _seen(q, n, window, sinks):
    """Keys that the queries of one sequence see together, and the sum of what each sees."""
    first = n - q
    pairs = 0
    for p in range(first, n):
        low = max(0, p - window + 1)
        pairs += p - low + 1 + min(low, sinks)
    low = max(0, first - window + 1)
    return n - low + min(low, sinks), pairs


def work(case):
    if case["op"] == "norm_rope":
        t = case["tokens"]
        return {"bytes": 2.0 * t * WIDTH * 2 + 4.0 * t, "flops": t * (HEADS + KV) * DIM * 8.0}
    if case["op"] == "window":
        seen = [_seen(q, n, case["window"], case["sinks"]) for q, n in zip(*_window_lengths(case))]
        rows = sum(_window_lengths(case)[0])
        return {"bytes": sum(k for k, _ in seen) * KV * DIM * 4.0 + rows * HEADS * DIM * 4.0,
                "flops": sum(p for _, p in seen) * HEADS * DIM * 4.0}
    sizes, prefix, suffix = _prefix_lengths(case)
    pairs = sum(m * p for m, p in zip(sizes, prefix)) + sum(suffix)
    return {"bytes": (sum(prefix) + sum(suffix)) * KV * DIM * 4.0 + case["batch"] * HEADS * DIM * 4.0,
            "flops": pairs * HEADS * DIM * 4.0}


# ---------------------------------------------------------------- inputs
def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _tables(chunks, seed):
    """A paged table: each list of logical chunks gets slots of one shuffled pool; what has been freed stays -1."""
    total = sum(len(c) for _, c in chunks)
    slots = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(chunks), max(1, max(m for m, _ in chunks))), -1, dtype=torch.int32)
    at = 0
    for b, (_, c) in enumerate(chunks):
        table[b, torch.tensor(c, dtype=torch.int64)] = slots[at: at + len(c)]
        at += len(c)
    return table, total


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "norm_rope":
        return _prepare_rope(case, seed, g)
    if case["op"] == "window":
        return _prepare_window(case, seed, g)
    return _prepare_prefix(case, seed, g)


def _prepare_rope(case, seed, g):
    t, half = case["tokens"], case["rot"] // 2
    s = {"op": "norm_rope", "layout": case["layout"], "rot": case["rot"], "scale": 1.0 + 0.1 * math.log(case["factor"])}
    s["qkv"] = _normal((t, WIDTH + case["pad"]), g)[:, :WIDTH]
    s["freq"] = (500000.0 ** -(torch.arange(half, device="cuda", dtype=torch.float64) / half) / case["factor"]).float()
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"] = 1 + 0.1 * torch.randn(DIM, generator=g, device="cuda")
        s["kw"] = 1 + 0.1 * torch.randn(DIM, generator=g, device="cuda")
    s["q"] = torch.empty((t, HEADS, DIM), device="cuda", dtype=torch.bfloat16)
    s["pool"] = case["pool"]
    r = random.Random(seed)
    if not case["pool"]:
        s["pos"] = torch.tensor([r.randrange(case["far"]) for _ in range(t)], dtype=torch.int32, device="cuda")
        s["k"] = torch.empty((t, KV, DIM), device="cuda", dtype=torch.bfloat16)
        s["v"] = torch.empty_like(s["k"])
        return s
    # Up to 64 tokens are one decode step, each of a sequence of its own; more are one prompt.
    step = t <= 64
    pos = [r.randrange(case["far"]) for _ in range(t)] if step else list(range(case["far"] - t, case["far"]))
    held = [(p // CHUNK + 1, [p // CHUNK]) for p in pos] if step else [
        (pos[-1] // CHUNK + 1, list(range(pos[0] // CHUNK, pos[-1] // CHUNK + 1)))]
    table, n = _tables(held, seed)
    s["table"] = table.cuda()
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    s["seq"] = torch.arange(t, dtype=torch.int32, device="cuda") if step else torch.zeros(t, dtype=torch.int32, device="cuda")
    s["k"] = _normal((n, KV, CHUNK, DIM), g)
    s["v"] = _normal((n, KV, CHUNK, DIM), g)
    return s


def _prepare_window(case, seed, g):
    q, n = _window_lengths(case)
    held = []
    for a, b in zip(q, n):
        low = max(0, b - a - case["window"] + 1) // CHUNK
        last = (b - 1) // CHUNK
        first = range(0, min(low, -(-case["sinks"] // CHUNK)))
        held.append((last + 1, list(first) + list(range(low, last + 1))))
    table, slots = _tables(held, seed)
    cu = [0]
    for a in q:
        cu.append(cu[-1] + a)
    s = {"op": "window", "window": case["window"], "sinks": case["sinks"], "max_q": max(q)}
    s["table"] = table.cuda()
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["len"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    # Where each query stands: what a scheduler has beside the offsets.
    s["row_seq"] = torch.tensor([b for b, a in enumerate(q) for _ in range(a)], device="cuda")
    s["row_at"] = torch.tensor([i for a in q for i in range(a)], device="cuda")
    s["k"] = _normal((slots, KV, CHUNK, DIM), g)
    s["v"] = _normal((slots, KV, CHUNK, DIM), g)
    s["q"] = _normal((cu[-1], HEADS, DIM), g)
    s["out"] = torch.empty((cu[-1], HEADS, DIM), device="cuda", dtype=torch.bfloat16)
    return s


def _prepare_prefix(case, seed, g):
    sizes, prefix, suffix = _prefix_lengths(case)
    held = [(-(-p // CHUNK), list(range(-(-p // CHUNK)))) for p in prefix + suffix]
    table, slots = _tables(held, seed)
    cu = [0]
    for m in sizes:
        cu.append(cu[-1] + m)
    most_p, most_s = (max(1, max(-(-x // CHUNK) for x in v)) for v in (prefix, suffix))
    s = {"op": "prefix", "prefix_table": table[: len(prefix), :most_p].contiguous().cuda(),
         "table": table[len(prefix):, :most_s].contiguous().cuda()}
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["prefix_len"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    s["suffix_len"] = torch.tensor(suffix, dtype=torch.int32, device="cuda")
    # Where each sequence stands in its group.
    s["group"] = torch.tensor([n for n, m in enumerate(sizes) for _ in range(m)], device="cuda")
    s["member"] = torch.tensor([i for m in sizes for i in range(m)], device="cuda")
    s["most"] = max(sizes)
    s["k"] = _normal((slots, KV, CHUNK, DIM), g)
    s["v"] = _normal((slots, KV, CHUNK, DIM), g)
    s["q"] = _normal((case["batch"], HEADS, DIM), g)
    s["out"] = torch.empty((case["batch"], HEADS, DIM), device="cuda", dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return {"norm_rope": _own_rope, "window": _own_window, "prefix": _own_prefix}[state["op"]](state)
    return {"norm_rope": _plain_rope, "window": _plain_window, "prefix": _plain_prefix}[state["op"]](state)


def _own_rope(s):
    import kv_chunk_selection_b200 as lsa
    inter = s["layout"] == "interleaved"
    if s["pool"]:
        lsa.lsa_qk_norm_rope_pool(s["qkv"], s["pos"], s["freq"], s["q"], s["k"], s["v"], s["table"], s["seq"], s["pos"],
                                  s["table"].shape[1], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=inter,
                                  rope_scale=s["scale"])
    else:
        lsa.lsa_qk_norm_rope(s["qkv"], s["pos"], s["freq"], s["q"], s["k"], s["v"], q_weight=s["qw"], k_weight=s["kw"],
                             eps=EPS, interleaved=inter, rope_scale=s["scale"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _own_window(s):
    import kv_chunk_selection_b200 as lsa
    if "workspace" not in s:
        s["workspace"] = lsa.new_window_attn_workspace(s["table"].shape[0], s["max_q"])
    lsa.lsa_window_attn(s["q"], s["k"], s["v"], s["table"], s["cu"], s["len"], s["table"].shape[1], s["max_q"], s["window"],
                        s["sinks"], s["out"], s["workspace"])
    return s["out"]


def _own_prefix(s):
    import kv_chunk_selection_b200 as lsa
    if "workspace" not in s:
        s["workspace"] = lsa.new_prefix_attn_workspace(s["table"].shape[0], s["prefix_table"].shape[0])
    lsa.lsa_prefix_decode_attn(s["q"], s["k"], s["v"], s["prefix_table"], s["cu"], s["prefix_len"], s["table"],
                               s["suffix_len"], s["out"], s["workspace"])
    return s["out"]


def _normed(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rotated(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, d), -1).flatten(-2) if interleaved else torch.cat((c, d), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(s):
    t, inter = s["qkv"].shape[0], s["layout"] == "interleaved"
    x = s["qkv"].float().view(t, HEADS + 2 * KV, DIM)
    angle = s["pos"].double()[:, None] * s["freq"].double()
    cos, sin = ((f(angle) * s["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    q = _rotated(_normed(x[:, :HEADS], s["qw"]), cos, sin, s["rot"], inter).to(torch.bfloat16)
    k = _rotated(_normed(x[:, HEADS: HEADS + KV], s["kw"]), cos, sin, s["rot"], inter).to(torch.bfloat16)
    v = x[:, HEADS + KV:].to(torch.bfloat16)
    if not s["pool"]:
        return {"q": q, "k": k, "v": v}
    slot, row = s["table"][s["seq"].long(), s["pos"].long() // CHUNK].long(), s["pos"].long() % CHUNK
    s["k"][slot, :, row] = k
    s["v"][slot, :, row] = v
    return {"q": q, "k": s["k"], "v": s["v"]}


def _plain_window(s):
    b, t, w, n = s["len"].shape[0], s["max_q"], s["window"], s["sinks"]
    length, cu = s["len"].long(), s["cu"].long()
    first = length - (cu[1:] - cu[:-1])                               # position of each sequence's first query
    near = first[:, None] - w + 1 + torch.arange(w + t - 1, device="cuda")
    sink = torch.arange(n, device="cuda").expand(b, n)
    at = torch.cat((sink, near), 1)                                   # positions of the keys: sinks, then all windows
    low = (first[:, None] - w + 1).clamp(min=0)
    held = torch.cat((sink < low, (near >= 0) & (near < length[:, None])), 1)
    at = torch.where(held, at, low.minimum(length[:, None] - 1))      # a held position in the place of the others
    slot = torch.gather(s["table"].long(), 1, at // CHUNK)
    k = s["k"][slot, :, at % CHUNK].float().permute(0, 2, 3, 1)       # [b, kv, dim, keys]
    v = s["v"][slot, :, at % CHUNK].float().transpose(1, 2)
    q = torch.zeros((b, t, HEADS, DIM), device="cuda")
    q[s["row_seq"], s["row_at"]] = s["q"].float()
    q = q.view(b, t, KV, GROUP, DIM).permute(0, 2, 3, 1, 4).reshape(b, KV, GROUP * t, DIM)
    score = (torch.matmul(q, k) / math.sqrt(DIM)).view(b, KV, GROUP, t, -1)
    p = first[:, None] + torch.arange(t, device="cuda")
    seen = held[:, None] & (at[:, None] <= p[:, :, None]) & ((at[:, None] > p[:, :, None] - w) | (at[:, None] < n))
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    weight = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    out = torch.matmul(weight.view(b, KV, GROUP * t, -1), v).view(b, KV, GROUP, t, DIM)
    out = out / weight.sum(-1, keepdim=True).clamp(min=1e-30)
    return out.permute(0, 3, 1, 2, 4).reshape(b, t, HEADS, DIM)[s["row_seq"], s["row_at"]].to(torch.bfloat16)


def _plain_prefix(s):
    groups, batch, m = s["prefix_len"].shape[0], s["suffix_len"].shape[0], s["most"]
    q = s["q"].float().view(batch, KV, GROUP, DIM)
    grouped = torch.zeros((groups, m, KV, GROUP, DIM), device="cuda")
    grouped[s["group"], s["member"]] = q
    tokens = lambda pool, table: pool[table.long().clamp(min=0)].float().transpose(1, 2).flatten(2, 3)  # noqa: E731
    kp, vp = tokens(s["k"], s["prefix_table"]), tokens(s["v"], s["prefix_table"])       # [groups, kv, tokens, dim]
    ks, vs = tokens(s["k"], s["table"]), tokens(s["v"], s["table"])                     # [batch, kv, tokens, dim]
    of_prefix = torch.matmul(grouped.transpose(1, 2).flatten(2, 3), kp.transpose(2, 3))
    of_prefix = of_prefix.view(groups, KV, m, GROUP, -1)[s["group"], :, s["member"]]    # [batch, kv, group, tokens]
    score = torch.cat((of_prefix, torch.matmul(q, ks.transpose(2, 3))), -1) / math.sqrt(DIM)
    there = torch.cat((torch.arange(kp.shape[2], device="cuda") < s["prefix_len"][s["group"]][:, None],
                       torch.arange(ks.shape[2], device="cuda") < s["suffix_len"][:, None]), 1)
    score = score.masked_fill(~there[:, None, None], -math.inf)
    weight = torch.exp(score - score.amax(-1, keepdim=True))
    weight = weight / weight.sum(-1, keepdim=True)
    back = torch.zeros((groups, m, KV, GROUP, kp.shape[2]), device="cuda")
    back[s["group"], s["member"]] = weight[..., : kp.shape[2]]
    out = torch.matmul(back.transpose(1, 2).flatten(2, 3), vp).view(groups, KV, m, GROUP, DIM)[s["group"], :, s["member"]]
    return (out + torch.matmul(weight[..., kp.shape[2]:], vs)).view(batch, HEADS, DIM).to(torch.bfloat16)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_rope(s)
    attend = _exact_window if case["op"] == "window" else _exact_prefix
    return attend(s)


def _exact_rope(s):
    x = s["qkv"].double()
    t, rot, inter = x.shape[0], s["rot"], s["layout"] == "interleaved"
    turn = torch.polar(torch.full((t, rot // 2), s["scale"], dtype=torch.float64, device="cuda"),
                       torch.outer(s["pos"].double(), s["freq"].double()))

    def head(h, weight):
        y = x[:, h * DIM: (h + 1) * DIM].clone()
        if weight is not None:
            y = y / torch.sqrt(y.square().sum(1, keepdim=True) / DIM + EPS) * weight.double()
        i = torch.arange(rot // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        z = torch.complex(y[:, a], y[:, b]) * turn
        y[:, a], y[:, b] = z.real, z.imag
        return y

    q = torch.stack([head(h, s["qw"]) for h in range(HEADS)], 1)
    k = torch.stack([head(HEADS + h, s["kw"]) for h in range(KV)], 1)
    v = x[:, (HEADS + KV) * DIM:].reshape(t, KV, DIM)
    if not s["pool"]:
        return {"q": q, "k": k, "v": v}
    kk, vv = s["k"].double(), s["v"].double()
    seq, pos, table = s["seq"].tolist(), s["pos"].tolist(), s["table"].tolist()
    slot = [table[b][p // CHUNK] for b, p in zip(seq, pos)]
    rows = torch.tensor([c * CHUNK + p % CHUNK for c, p in zip(slot, pos)], device="cuda")
    for pool, new in ((kk, k), (vv, v)):
        for h in range(KV):
            flat = pool[:, h].reshape(-1, DIM)
            flat[rows] = new[:, h]
            pool[:, h] = flat.view(-1, CHUNK, DIM)
    return {"q": q, "k": kk, "v": vv}


def _attended(q, k, v, seen):
    """softmax(q k^T / sqrt(d)) v over the seen keys, for one KV head; q [rows, group, dim]."""
    score = torch.einsum("rgd,kd->grk", q, k) / DIM ** 0.5
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    return torch.einsum("grk,kd->rgd", torch.softmax(score, -1), v)


def _rows(pool, slots, h, n):
    return pool[slots, h].reshape(-1, DIM)[:n].double()


def _exact_window(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, n = s["cu"].tolist(), s["len"].tolist()
    for b in range(len(n)):
        p = torch.arange(n[b] - (cu[b + 1] - cu[b]), n[b], device="cuda")[:, None]
        alive = torch.nonzero(s["table"][b] >= 0)[:, 0].tolist()
        slots = s["table"][b, alive].long()
        j = (torch.tensor(alive, device="cuda")[:, None] * CHUNK + torch.arange(CHUNK, device="cuda")).reshape(1, -1)
        seen = (j <= p) & ((p - j < s["window"]) | (j < s["sinks"]))
        for h in range(KV):
            at = slice(h * GROUP, (h + 1) * GROUP)
            k, v = _rows(s["k"], slots, h, None), _rows(s["v"], slots, h, None)
            for r in range(cu[b], cu[b + 1], 1024):
                e = min(r + 1024, cu[b + 1])
                out[r:e, at] = _attended(s["q"][r:e, at].double(), k, v, seen[r - cu[b]: e - cu[b]])
    return out


def _exact_prefix(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, n, m = s["cu"].tolist(), s["prefix_len"].tolist(), s["suffix_len"].tolist()
    for g in range(len(n)):
        for h in range(KV):
            at = slice(h * GROUP, (h + 1) * GROUP)
            kp, vp = (_rows(s[x], s["prefix_table"][g, : -(-n[g] // CHUNK)].long(), h, n[g]) for x in ("k", "v"))
            for b in range(cu[g], cu[g + 1]):
                ks, vs = (_rows(s[x], s["table"][b, : -(-m[b] // CHUNK)].long(), h, m[b]) for x in ("k", "v"))
                k, v = torch.cat((kp, ks)), torch.cat((vp, vs))
                out[b: b + 1, at] = _attended(s["q"][b: b + 1, at].double(), k, v, torch.ones((), dtype=torch.bool, device="cuda"))
    return out
