"""The operators around the paged context cache, as measured cases.

Four operators, of one layer of the draft each, over the paged bf16 cache
[num_blocks, H, block_size, 128] that `context_kv_store` fills:

rotary     rotary positions: the cos/sin table with its scalings for long
           contexts (`rope_table`), and the rotation of query heads, or of
           their gradients, by that table (`rope_rotate`)
attention  drafted tokens (one, a chain, or a tree given by an ancestor mask)
           attending to their sequence's cached context and to each other
           (`context_tree_attention`)
mass       the attention weight each cached cell has received, summed over the
           queries (`context_attention_mass`)
evict      keeping the `budget` cells of every head with the most weight
           (`context_kv_evict`)

`run` computes a case in elementary torch operations, or with `own` by the
framework's entry points.
"""

import math
import random

import numpy as np
import torch

own = False

HEAD = 64  # the cache's head width: K in the first 64 of 128 elements, V in the rest

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one drafting step's queries: 16 rows, 64 query heads, pairs as the store rotates its keys
        dict(name="rotate-step", op="rotary", kind="rotate", tokens=16, heads=64, head_dim=64, rotary_dim=64,
             max_position=16384, layout="interleaved", inverse=False, type="bf16", table="bf16"),
        # a long prompt's queries in the half layout, FP32 table
        dict(name="rotate-prompt", op="rotary", kind="rotate", tokens=16384, heads=64, head_dim=64, rotary_dim=64,
             max_position=131072, layout="half", inverse=False, type="bf16", table="fp32"),
        # the gradient (the inverse rotation) of a partly rotated wide head, a ragged number of rows
        dict(name="rotate-gradient", op="rotary", kind="rotate", tokens=4099, heads=24, head_dim=128, rotary_dim=64,
             max_position=32768, layout="interleaved", inverse=True, type="fp16", table="fp32"),
        # the whole table of a context stretched eightfold, built at start-up or when the stretch changes
        dict(name="table-stretched", op="rotary", kind="table", count=131072, start=0, rotary_dim=64, width=64,
             base=500000.0, scaling="ramp", factor=8.0, original_max=16384, low=1.0, high=32.0, magnitude=1.2,
             table="bf16"),
        # one token of one short sequence: the smallest call, latency alone
        dict(name="attend-one", op="attention", batch=1, heads=8, group=8, nodes=1, max_ctx=1000, block_size=16,
             tree=False, softcap=0.0, lens_seed=1),
        # a serving batch at one token per sequence, ragged contexts
        dict(name="attend-batch", op="attention", batch=64, heads=8, group=8, nodes=1, max_ctx=8192, block_size=16,
             tree=False, softcap=0.0, lens_seed=2),
        # verification of drafted trees: ragged trees and contexts, odd pages and groups
        dict(name="attend-trees", op="attention", batch=16, heads=2, group=5, nodes=33, max_ctx=4096, block_size=24,
             tree=True, softcap=0.0, lens_seed=3),
        # large trees over long contexts with capped scores: the largest call
        dict(name="attend-long", op="attention", batch=4, heads=8, group=8, nodes=64, max_ctx=65536, block_size=16,
             tree=True, softcap=30.0, lens_seed=4),
        # the weights of one verification step of one sequence
        dict(name="mass-step", op="mass", batch=1, heads=8, group=8, nodes=8, max_ctx=2048, block_size=16,
             tree=True, softcap=0.0, decay=1.0, lens_seed=5),
        # the same for a batch of large trees, with decay
        dict(name="mass-batch", op="mass", batch=16, heads=8, group=8, nodes=64, max_ctx=16384, block_size=16,
             tree=True, softcap=0.0, decay=0.98, lens_seed=6),
        # the steady state of a capped cache: a few tokens over the budget, every sequence of the batch
        dict(name="evict-steady", op="evict", batch=32, heads=8, max_len=4160, budget=4096, block_size=16, sinks=4,
             recent=128, lens_seed=7),
        # a long prompt cut to half
        dict(name="evict-long", op="evict", batch=2, heads=8, max_len=65536, budget=32768, block_size=16, sinks=4,
             recent=256, lens_seed=8),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotary", "attention", "attention", "mass", "evict"])
    if op == "rotary" and rng.random() < 0.3:
        scaling = rng.choice(["none", "linear", "base", "bands", "ramp"])
        rotary = 2 * rng.randint(2, 64)
        return dict(op="rotary", kind="table", count=_log(rng, 16, 131072), start=_log(rng, 1, 100000) - 1,
                    rotary_dim=rotary, width=rotary + 2 * rng.choice([0, 0, 3, 16]),
                    base=rng.choice([10000.0, 500000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.uniform(1.5, 16.0), original_max=_log(rng, 1024, 32768),
                    low=1.0, high=rng.choice([4.0, 32.0]), magnitude=rng.choice([1.0, 1.1]),
                    table=rng.choice(["bf16", "fp32"]))
    if op == "rotary":
        head = rng.choice([64, 64, 96, 128, 80])
        rotary = rng.choice([head, head, head // 2, head // 4])
        heads = rng.choice([1, 5, 8, 24, 64])
        return dict(op="rotary", kind="rotate", tokens=_log(rng, 1, (1 << 26) // (heads * head)), heads=heads,
                    head_dim=head, rotary_dim=rotary, max_position=_log(rng, 1024, 131072),
                    layout=rng.choice(["interleaved", "half"]), inverse=rng.random() < 0.4,
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), table=rng.choice(["bf16", "fp32"]))
    if op == "evict":
        heads, batch = rng.choice([1, 2, 8, 16]), _log(rng, 1, 32)
        longest = _log(rng, 32, max(32, min(65536, (1 << 20) // (heads * batch))))
        budget = max(1, int(longest * rng.choice([0.98, 0.9, 0.5, rng.uniform(0.05, 1.0)])))
        return dict(op="evict", batch=batch, heads=heads, max_len=longest, budget=budget,
                    block_size=rng.choice([1, 16, 16, 24, 64]), sinks=rng.choice([0, 4]),
                    recent=rng.choice([0, 8, budget // 4]), lens_seed=rng.randrange(1 << 30))
    heads, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 5, 8])
    batch, nodes, ctx = _log(rng, 1, 64), _log(rng, 1, 100), _log(rng, 1, 65536)
    while batch * heads * ctx > 1 << 21 or batch * heads * group * nodes * ctx > 1 << 28:
        ctx = max(1, ctx // 2 + rng.randint(0, 1))
        batch = max(1, batch - batch // 3)
    case = dict(op=op, batch=batch, heads=heads, group=group, nodes=nodes, max_ctx=ctx,
                block_size=rng.choice([8, 16, 16, 24, 64]), tree=rng.random() < 0.7,
                softcap=rng.choice([0.0, 0.0, 30.0]), lens_seed=rng.randrange(1 << 30))
    if op == "mass":
        case["decay"] = rng.choice([1.0, 0.98])
    return case


def _lens(case):
    """The sequences' context lengths and drafted tokens: the first is the longest, the others ragged."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "evict":
        low = case["max_len"] - case["max_len"] // 64 if case["budget"] * 10 > case["max_len"] * 9 else 1
        return [case["max_len"]] + [rng.randint(low, case["max_len"]) for _ in range(case["batch"] - 1)], None
    ctx = [case["max_ctx"]] + [rng.randint(max(1, case["max_ctx"] // 4), case["max_ctx"])
                               for _ in range(case["batch"] - 1)]
    nodes = [case["nodes"]] + [rng.randint(max(1, case["nodes"] // 2), case["nodes"])
                               for _ in range(case["batch"] - 1)]
    return ctx, nodes


def _size(name):
    return 4 if name == "fp32" else 2


def work(case):
    if case["op"] == "rotary":
        if case["kind"] == "table":
            n = case["count"] * case["width"]
            return {"bytes": n * _size(case["table"]), "flops": 4 * n}
        n = case["tokens"] * case["heads"] * case["head_dim"]
        turned = case["tokens"] * case["heads"] * case["rotary_dim"]
        rows = min(case["tokens"], case["max_position"])
        return {"bytes": 2 * n * _size(case["type"]) + rows * case["rotary_dim"] * _size(case["table"]) +
                8 * case["tokens"], "flops": 3 * turned}
    lens, nodes = _lens(case)
    H = case["heads"]
    if case["op"] == "evict":
        total, moved, kept = 0, 0, 0
        for n in lens:
            keep = min(n, case["budget"])
            total += n
            kept += case["budget"]
            moved += keep * (n - keep) // n  # the evicted cells among the first `keep`, for weights in any order
        return {"bytes": H * (8 * total + 8 * kept + 2 * 4 * HEAD * moved), "flops": 4 * H * total}
    G = case["group"]
    keys = sum(c + n for c, n in zip(lens, nodes))
    rows = sum(nodes) * H * G
    pairs = sum((c + n) * n for c, n in zip(lens, nodes)) * H * G
    if case["op"] == "attention":
        return {"bytes": keys * H * 4 * HEAD + rows * (4 * HEAD + 4), "flops": 4 * HEAD * pairs}
    cells = case["batch"] * H * (case["max_ctx"] + case["nodes"])
    return {"bytes": keys * H * 2 * HEAD + rows * (2 * HEAD + 4) + 8 * cells, "flops": 2 * HEAD * pairs}


def _tree_words(case, counts, rng):
    """Ancestor masks of random trees, int64 [sum of nodes, words]: bit j of row i is set if node j is node i or
    one of the nodes above it."""
    words = (case["nodes"] + 63) // 64
    rows = []
    for n in counts:
        seen = []
        for i in range(n):
            parent = rng.randrange(max(0, i - 8), i) if i else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        rows += [[(s >> 64 * w) & 0xFFFFFFFFFFFFFFFF for w in range(words)] for s in seen]
    return torch.from_numpy(np.array(rows, dtype=np.uint64).view(np.int64).reshape(len(rows), words))


def _pages(lens, block_size, gen):
    """A pool with each sequence's pages scattered over it: block tables int32 [B, widest] and the pool's size."""
    counts = [(n + block_size - 1) // block_size for n in lens]
    total = sum(counts)
    order = torch.randperm(total, generator=gen).to(torch.int32)
    tables = torch.zeros(len(lens), max(counts), dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        tables[b, :c] = order[at:at + c]
        at += c
    return tables, total


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t.normal_(0.0, scale, generator=gen)

    if case["op"] == "rotary":
        if case["kind"] == "table":
            # other seeds: a base a little off, as a stretched context picks its own
            return dict(case, base=case["base"] * (1.0 + (seed % 1009) * 1e-4), device=dev)
        table = _table(dict(count=case["max_position"], start=0, rotary_dim=case["rotary_dim"],
                            width=case["rotary_dim"], base=10000.0, scaling="none", factor=1.0, original_max=1,
                            low=1.0, high=2.0, magnitude=1.0, table=case["table"], device=dev))
        positions = torch.randint(0, case["max_position"], (case["tokens"],), generator=gen, device=dev)
        return dict(case, x=normal(case["tokens"], case["heads"], case["head_dim"], dtype=TYPES[case["type"]]),
                    positions=positions, cos_sin=table)

    lens, nodes = _lens(case)
    H, bs = case["heads"], case["block_size"]
    if case["op"] == "evict":
        tables, blocks = _pages(lens, bs, host)
        # weights summed over many queries: over some orders of magnitude, a few cells never seen
        weights = torch.exp(2.0 * normal(case["batch"], H, case["max_len"], dtype=torch.float32))
        weights[torch.rand(weights.shape, generator=gen, device=dev) < 0.01] = 0.0
        at = torch.arange(case["max_len"], dtype=torch.int32, device=dev)
        return dict(case, cache=normal(blocks, H, bs, 2 * HEAD), tables=tables.to(dev),
                    lens=torch.tensor(lens, dtype=torch.int32, device=dev), weights=weights,
                    positions=at.expand(case["batch"], H, -1).contiguous(),
                    ends=torch.tensor(lens, dtype=torch.int32, device=dev))
    G, T = case["group"], sum(nodes)
    tables, blocks = _pages([c + n for c, n in zip(lens, nodes)], bs, host)
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    state = dict(case, q=normal(T, H * G, HEAD, scale=2.0), cache=normal(blocks, H, bs, 2 * HEAD),
                 tables=tables.to(dev), ctx_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                 q_starts=torch.tensor(starts, dtype=torch.int32, device=dev),
                 tree_mask=_tree_words(case, nodes, rng).to(dev) if case["tree"] else None)
    if case["op"] == "mass":
        state["width"] = case["max_ctx"] + case["nodes"]
        state["lse"] = _lse(state)
        state["weights"] = torch.rand(case["batch"], H, state["width"], generator=gen, device=dev)
    return state


# ---- rotary -------------------------------------------------------------------------------------------------------

def _frequencies(s):
    """Turns per position of every pair, in 64 bits: base^(-2 j / R), scaled."""
    R, half = s["rotary_dim"], s["rotary_dim"] // 2
    j = torch.arange(half, dtype=torch.float64)
    base = s["base"]
    if s["scaling"] == "base":
        base = base * s["factor"] ** (R / (R - 2))
    f = base ** (-2.0 * j / R)
    if s["scaling"] == "linear":
        f = f / s["factor"]
    elif s["scaling"] == "bands":
        turns = s["original_max"] * f / (2.0 * math.pi)
        t = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0.0, 1.0)
        f = f * ((1.0 - t) / s["factor"] + t)
    elif s["scaling"] == "ramp":
        def index(turns):
            return R * math.log(s["original_max"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(s["base"]))
        lo, hi = max(0.0, math.floor(index(s["high"]))), min(half - 1.0, math.ceil(index(s["low"])))
        t = ((j - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f * (t / s["factor"] + (1.0 - t))
    return f


def _table(s):
    """[count, width]: cos of the width / 2 pairs, then their sin; pairs past the rotary ones do not turn."""
    f = _frequencies(s).to(s["device"])
    at = torch.arange(s["start"], s["start"] + s["count"], dtype=torch.float64, device=s["device"])
    angle = at[:, None] * f[None, :]
    rest = (s["width"] - s["rotary_dim"]) // 2
    ones = torch.ones(s["count"], rest, dtype=torch.float64, device=s["device"])
    return torch.cat([torch.cos(angle) * s["magnitude"], ones, torch.sin(angle) * s["magnitude"],
                      torch.zeros_like(ones)], dim=1).to(TYPES[s["table"]])


def _pairs(x, R, layout):
    return (x[..., 0:R:2], x[..., 1:R:2]) if layout == "interleaved" else (x[..., :R // 2], x[..., R // 2:R])


def _rotate(s):
    R = s["rotary_dim"]
    x = s["x"].float()
    row = s["cos_sin"][s["positions"]].float()[:, None, :]
    c, n = row[..., :R // 2], row[..., R // 2:]
    if s["inverse"]:
        n = -n
    a, b = _pairs(x, R, s["layout"])
    first, second = a * c - b * n, b * c + a * n
    turned = (torch.stack([first, second], dim=-1).flatten(-2) if s["layout"] == "interleaved"
              else torch.cat([first, second], dim=-1))
    return torch.cat([turned, x[..., R:]], dim=-1).to(s["x"].dtype)


# ---- attention ----------------------------------------------------------------------------------------------------

def _scores(s, seq):
    """Of the sequences `seq` (a slice): scores [b, H, nodes, G, keys] in 32 bits with what each may see, the rows'
    query indexes, which of them there are, and the cached values."""
    H, G, n, bs = s["heads"], s["group"], s["nodes"], s["block_size"]
    dev = s["q"].device
    starts, ctx = s["q_starts"].long(), s["ctx_lens"].long()[seq]
    first, count = starts[:-1][seq], (starts[1:] - starts[:-1])[seq]
    node = torch.arange(n, device=dev)
    rows = (first[:, None] + node).clamp(max=s["q"].shape[0] - 1)
    live = node < count[:, None]
    key = torch.arange(s["max_ctx"] + n, device=dev)
    block = (key // bs).clamp(max=s["tables"].shape[1] - 1)
    cells = s["cache"][s["tables"][seq].long()[:, block], :, key % bs]  # [b, keys, H, 128]
    cells = cells.float().permute(0, 2, 1, 3)
    q = s["q"][rows].float().view(-1, n, H, G, HEAD).permute(0, 2, 1, 3, 4).reshape(-1, H, n * G, HEAD)
    score = torch.matmul(q, cells[..., :HEAD].transpose(2, 3).contiguous()).view(-1, H, n, G, key.numel())
    score = score * 0.125
    if s["softcap"]:
        score = s["softcap"] * torch.tanh(score / s["softcap"])
    other = key - ctx[:, None]  # the node that a key holds, negative for the context
    if s["tree_mask"] is None:
        sees = other[:, None, :] <= node[None, :, None]
    else:
        words = s["tree_mask"][rows]  # [b, nodes, words]
        at = other.clamp(0, 64 * words.shape[2] - 1)[:, None, :].expand(-1, n, -1)
        sees = (torch.gather(words, 2, at // 64) >> (at % 64)) & 1 == 1
        sees = sees & (other < count[:, None])[:, None, :] | (other < 0)[:, None, :]
    sees = sees & live[:, :, None]
    return score.masked_fill(~sees[:, None, :, None, :], -math.inf), rows, live, cells[..., HEAD:]


def _each(s, limit=1 << 29):
    """Slices of the batch whose scores fit `limit`."""
    one = s["heads"] * s["group"] * s["nodes"] * (s["max_ctx"] + s["nodes"])
    step = max(1, limit // one)
    return [slice(b, min(b + step, s["batch"])) for b in range(0, s["batch"], step)]


def _softmax(score):
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    return p, total, (top + torch.log(total)).squeeze(-1)


def _scatter(out, value, rows, live):
    """value [b, H, nodes, G, ...] to rows of out [T, H G, ...]; rows past a sequence's nodes go to a spare last row."""
    at = torch.where(live, rows, torch.full_like(rows, out.shape[0] - 1)).flatten()
    value = value.transpose(1, 2).flatten(2, 3).flatten(0, 1)
    out.index_copy_(0, at, value.to(out.dtype))


def _attention(s):
    T, heads = s["q"].shape[:2]
    out = torch.empty(T + 1, heads, HEAD, dtype=torch.bfloat16, device=s["q"].device)
    lse = torch.empty(T + 1, heads, dtype=torch.float32, device=s["q"].device)
    for seq in _each(s):
        score, rows, live, v = _scores(s, seq)
        p, total, logsum = _softmax(score)
        b, H, n, G, keys = p.shape
        o = torch.matmul(p.view(b, H, n * G, keys), v.contiguous()).view(b, H, n, G, HEAD)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        _scatter(out, o, rows, live)
        _scatter(lse, logsum, rows, live)
    return out[:T], lse[:T]


def _lse(s):
    T, heads = s["q"].shape[:2]
    lse = torch.empty(T + 1, heads, dtype=torch.float32, device=s["q"].device)
    for seq in _each(s):
        score, rows, live, _ = _scores(s, seq)
        _scatter(lse, _softmax(score)[2], rows, live)
    return lse[:T].contiguous()


def _mass(s):
    out = torch.empty_like(s["weights"])
    for seq in _each(s):
        score, rows, live, _ = _scores(s, seq)
        b, H, n, G, keys = score.shape
        lse = s["lse"][rows].view(b, n, H, G).transpose(1, 2)[..., None]
        p = torch.where(score == -math.inf, torch.zeros_like(score), torch.exp(score - lse))
        mass = p.sum(dim=(2, 3))
        total = s["ctx_lens"].long()[seq] + (s["q_starts"][1:] - s["q_starts"][:-1]).long()[seq]
        there = torch.arange(keys, device=mass.device) < total[:, None, None]
        out[seq] = torch.where(there, s["weights"][seq] * s["decay"] + mass, torch.zeros_like(mass))
    return out


# ---- eviction -----------------------------------------------------------------------------------------------------

def _evict(s):
    W, budget, bs, H = s["max_len"], s["budget"], s["block_size"], s["heads"]
    B, dev = s["batch"], s["cache"].device
    at = torch.arange(W, device=dev)
    size = s["lens"].long()[:, None, None]
    there = at < size
    # the order of keeping: the protected, then by weight (a NaN as the least), the first of equals first
    key = torch.nan_to_num(s["weights"].double(), nan=-1e300, posinf=1e300, neginf=-1e300)
    old = (s["positions"] < s["sinks"]) | (s["positions"] >= (s["ends"] - s["recent"])[:, None, None])
    key = torch.where(old, math.inf, key)
    key = torch.where(there, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept_count = size.clamp(max=budget)
    keep = torch.zeros_like(there.expand(B, H, W)).contiguous()
    keep.scatter_(2, order, (at < kept_count).expand(B, H, W))
    # kept cells past the new end fill the holes before it, both in rising order
    hole = ~keep & (at < kept_count)
    far = keep & (at >= kept_count)
    far_rank = torch.where(far, far.cumsum(-1) - 1, torch.full_like(order, W))
    source = torch.zeros(B, H, W + 1, dtype=torch.int64, device=dev)
    source.scatter_(2, far_rank, at.expand(B, H, W))
    hole_rank = (hole.cumsum(-1) - 1).clamp(min=0)
    origin = torch.where(hole, torch.gather(source, 2, hole_rank), at.expand(B, H, W))[..., :budget]
    there = (torch.arange(budget, device=dev) < kept_count).expand(B, H, budget)
    weights = torch.where(there, torch.gather(s["weights"], 2, origin), 0.0)
    positions = torch.where(there, torch.gather(s["positions"], 2, origin), -1)
    # cells past the new end stay, so they are written with themselves; past the table they fall on its last page's
    b, h = torch.arange(B, device=dev)[:, None, None], torch.arange(H, device=dev)[None, :, None]
    tables = s["tables"].long()
    to = torch.where(there, torch.arange(budget, device=dev), 0)
    origin = torch.where(there, origin, origin[..., :1])
    cells = s["cache"][tables[b, origin // bs], h, origin % bs]
    s["cache"][tables[b, to // bs], h, to % bs] = cells
    return weights, positions, s["lens"].clamp(max=budget), s["cache"]


# ---- one pass -----------------------------------------------------------------------------------------------------

def _own(s):
    import norm_rope_cache_amd as nrc

    if s["op"] == "rotary":
        if s["kind"] == "table":
            return nrc.rope_table(s["count"], s["rotary_dim"], base=s["base"], scaling=s["scaling"],
                                  factor=s["factor"], original_max=s["original_max"], low=s["low"], high=s["high"],
                                  magnitude=s["magnitude"], width=s["width"], start=s["start"],
                                  dtype=TYPES[s["table"]], device=s["device"])
        return nrc.rope_rotate(s["x"], s["positions"], s["cos_sin"], layout=s["layout"], inverse=s["inverse"])
    if s["op"] == "attention":
        return nrc.context_tree_attention(s["q"], s["cache"], s["tables"], s["ctx_lens"], s["q_starts"], s["nodes"],
                                          max_ctx=s["max_ctx"], tree_mask=s["tree_mask"], softcap=s["softcap"])
    if s["op"] == "mass":
        return nrc.context_attention_mass(s["q"], s["cache"], s["tables"], s["ctx_lens"], s["q_starts"], s["lse"],
                                          s["nodes"], tree_mask=s["tree_mask"], softcap=s["softcap"],
                                          weights=s["weights"], decay=s["decay"])
    weights, positions, lens = nrc.context_kv_evict(s["cache"], s["tables"], s["lens"], s["weights"], s["positions"],
                                                    s["ends"], s["budget"], sinks=s["sinks"], recent=s["recent"])
    return weights, positions, lens, s["cache"]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "rotary":
        return _table(state) if state["kind"] == "table" else _rotate(state)
    return {"attention": _attention, "mass": _mass, "evict": _evict}[state["op"]](state)


# ---- 64 bits ------------------------------------------------------------------------------------------------------

def _exact_scores(s, b, h, sees):
    """Scores of sequence b's queries on KV head h over its own keys, 64 bits: [nodes, G, keys], unseen -inf."""
    G, bs = s["group"], s["block_size"]
    lo, hi = (int(v) for v in s["q_starts"][b:b + 2])
    keys = int(s["ctx_lens"][b]) + hi - lo
    page = s["tables"][b].long()[torch.arange(keys, device=s["q"].device) // bs]
    cell = s["cache"][page, h, torch.arange(keys, device=s["q"].device) % bs].double()
    q = s["q"][lo:hi, h * G:(h + 1) * G].double().reshape(-1, HEAD)
    score = (q @ cell[:, :HEAD].T.contiguous()).reshape(hi - lo, G, keys) / 8.0
    if s["softcap"]:
        score = torch.tanh(score / s["softcap"]) * s["softcap"]
    return score.masked_fill(~sees[:, None, :], -math.inf), cell[:, HEAD:]


def _exact_sees(s, b):
    lo, hi = (int(v) for v in s["q_starts"][b:b + 2])
    ctx, n = int(s["ctx_lens"][b]), hi - lo
    sees = np.ones((n, ctx + n), dtype=bool)
    if s["tree_mask"] is None:
        sees[:, ctx:] = np.tril(np.ones((n, n), dtype=bool))
    else:
        words = s["tree_mask"][lo:hi].cpu().numpy().view(np.uint8)
        sees[:, ctx:] = np.unpackbits(words, axis=1, bitorder="little")[:, :n].astype(bool)
    return torch.from_numpy(sees).to(s["q"].device)


def exact(case, seed):
    if case["op"] == "evict":
        return None  # values are moved, none is computed
    s = prepare(case, seed)
    if case["op"] == "rotary" and case["kind"] == "table":
        # one pair at a time, by the definition, on the host
        R, half = s["rotary_dim"], s["width"] // 2
        at = np.arange(s["start"], s["start"] + s["count"], dtype=np.float64)
        out = np.zeros((s["count"], s["width"]))
        out[:, R // 2:half] = 1.0
        base = s["base"] * (s["factor"] ** (R / (R - 2.0)) if s["scaling"] == "base" else 1.0)
        for j in range(R // 2):
            f = math.exp(-2.0 * j / R * math.log(base))
            turns = s["original_max"] * f / (2.0 * math.pi)
            if s["scaling"] == "linear":
                f /= s["factor"]
            elif s["scaling"] == "bands":
                t = (turns - s["low"]) / (s["high"] - s["low"])
                f = f if t >= 1 else f / s["factor"] if t <= 0 else f * (t + (1.0 - t) / s["factor"])
            elif s["scaling"] == "ramp":
                per = R / (2.0 * math.log(s["base"]))
                lo = max(0.0, math.floor(per * math.log(s["original_max"] / (s["high"] * 2.0 * math.pi))))
                hi = min(R // 2 - 1.0, math.ceil(per * math.log(s["original_max"] / (s["low"] * 2.0 * math.pi))))
                t = min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3)))
                f = f * (1.0 - t) + f / s["factor"] * t
            out[:, j] = s["magnitude"] * np.cos(at * f)
            out[:, half + j] = s["magnitude"] * np.sin(at * f)
        return out
    if case["op"] == "rotary":
        # each pair as a complex number, turned by its angle's
        R = s["rotary_dim"]
        x = s["x"].double()
        row = s["cos_sin"].double()[s["positions"]]
        turn = torch.complex(row[:, :R // 2], row[:, R // 2:])[:, None, :]
        if s["inverse"]:
            turn = turn.conj()
        a, b = _pairs(x, R, s["layout"])
        y = torch.complex(a.contiguous(), b.contiguous()) * turn
        out = x.clone()
        u, v = _pairs(out, R, s["layout"])
        u.copy_(y.real)
        v.copy_(y.imag)
        return out
    T, heads = s["q"].shape[:2]
    dev, H, G = s["q"].device, s["heads"], s["group"]
    if case["op"] == "attention":
        out = torch.zeros(T, heads, HEAD, dtype=torch.float64, device=dev)
        lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device=dev)
        for b in range(s["batch"]):
            lo, hi = (int(v) for v in s["q_starts"][b:b + 2])
            sees = _exact_sees(s, b)
            for h in range(H):
                score, v = _exact_scores(s, b, h, sees)
                l = torch.logsumexp(score, dim=-1)
                p = torch.exp(score - l[..., None])
                o = p.reshape(-1, p.shape[-1]) @ v
                out[lo:hi, h * G:(h + 1) * G] = o.reshape(hi - lo, G, HEAD)
                lse[lo:hi, h * G:(h + 1) * G] = l
        return out, lse
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device=dev)
    for b in range(s["batch"]):
        lo, hi = (int(v) for v in s["q_starts"][b:b + 2])
        sees = _exact_sees(s, b)
        for h in range(H):
            score, _ = _exact_scores(s, b, h, sees)
            p = torch.exp(score - s["lse"][lo:hi, h * G:(h + 1) * G].double()[..., None])
            keys = score.shape[-1]
            out[b, h, :keys] = p.sum(dim=(0, 1)) + s["weights"][b, h, :keys].double() * s["decay"]
    return out
