"""Operators of a drafted token's way to the context cache, as measured cases.

prepare    norms of queries and keys for each head with the rotation in the same
           pass (`qk_norm_rotate`), and its gradient (`qk_norm_rotate_grad`)
pack       K and V rows into the cells of a 4-bit paged cache and back
           (`context_fp4_store`, `context_fp4_load`)
fp4        drafted tokens (one, a chain, a tree) attending to a cache held in
           4 bits (`context_fp4_attention`)
window     the same over the bf16 cache with a sliding window and a few first
           tokens that stay visible (`context_window_attention`)

A 4-bit cache is uint8 [num_blocks, H, page_bytes]. A page of a head holds, for
its block_size cells, 32 bytes of K codes each, then 32 bytes of V codes each, then
4 scale bytes each (K's two groups of 32 elements, V's two), rounded up to 16 bytes.
An element is its code's value (sign, 0 .5 1 1.5 2 3 4 6; the even element in the low
half of the byte) times 2^(scale byte - 127); a group's exponent is the least with
which no element passes 6, held to -120 .. 125.

`run` computes a case in elementary torch operations, or with `own` by the
framework's entry points.
"""

import math
import random

import numpy as np
import torch

own = False

HEAD = 64  # the caches' head width

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one drafting step: 16 rows of 64 query heads and 8 key heads, without gains, as the chain's own keys
        dict(name="prepare-step", op="prepare", grad=False, tokens=16, q_heads=64, k_heads=8, head_dim=64, rotary_dim=64,
             max_position=16384, layout="interleaved", type="bf16", weight="none", table="bf16"),
        # a long prompt in the half layout, with gains
        dict(name="prepare-prompt", op="prepare", grad=False, tokens=16384, q_heads=64, k_heads=8, head_dim=64,
             rotary_dim=64, max_position=131072, layout="half", type="bf16", weight="bf16", table="fp32"),
        # training: the gradients of partly rotated wide heads, a ragged number of rows
        dict(name="prepare-gradient", op="prepare", grad=True, tokens=4099, q_heads=24, k_heads=3, head_dim=128,
             rotary_dim=64, max_position=32768, layout="interleaved", type="fp16", weight="fp32", table="fp32"),
        # training: the gradients of a whole packed batch
        dict(name="prepare-gradient-long", op="prepare", grad=True, tokens=16384, q_heads=64, k_heads=8, head_dim=64,
             rotary_dim=64, max_position=131072, layout="half", type="bf16", weight="bf16", table="bf16"),
        # the drafted tokens of a step into the cells of 4 layers
        dict(name="pack-step", op="pack", layers=4, tokens=33, heads=8, block_size=16, skipped=0.06),
        # a prompt's context into the cells of 4 layers
        dict(name="pack-prompt", op="pack", layers=4, tokens=8197, heads=8, block_size=16, skipped=0.0),
        # one token of one short sequence: latency alone
        dict(name="fp4-one", op="fp4", batch=1, heads=8, group=8, nodes=1, max_ctx=1000, block_size=16, tree=False,
             softcap=0.0, window=0, sinks=0, lens_seed=1),
        # a serving batch at one token per sequence, ragged contexts
        dict(name="fp4-batch", op="fp4", batch=64, heads=8, group=8, nodes=1, max_ctx=16384, block_size=16, tree=False,
             softcap=0.0, window=0, sinks=0, lens_seed=2),
        # verification of large drafted trees over long contexts
        dict(name="fp4-trees", op="fp4", batch=4, heads=8, group=8, nodes=48, max_ctx=65536, block_size=64, tree=True,
             softcap=0.0, window=0, sinks=0, lens_seed=3),
        # a chain of five drafted tokens far into one sequence, odd pages
        dict(name="window-one", op="window", batch=1, heads=8, group=5, nodes=5, max_ctx=32768, block_size=24,
             tree=False, softcap=0.0, window=1024, sinks=4, lens_seed=4),
        # a serving batch behind a window
        dict(name="window-batch", op="window", batch=64, heads=8, group=8, nodes=1, max_ctx=16384, block_size=16,
             tree=False, softcap=0.0, window=4096, sinks=4, lens_seed=5),
        # two prompts' chunks of 4096 tokens behind a window
        dict(name="window-prompt", op="window", batch=2, heads=8, group=8, nodes=4096, max_ctx=8192, block_size=16,
             tree=False, softcap=0.0, window=1024, sinks=4, lens_seed=6),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prepare", "prepare", "pack", "fp4", "fp4", "window", "window"])
    if op == "prepare":
        head = rng.choice([64, 64, 96, 128, 80, 256])
        q_heads, k_heads = rng.choice([(1, 1), (8, 1), (24, 8), (5, 5), (64, 8)])
        return dict(op=op, grad=rng.random() < 0.5, tokens=_log(rng, 1, (1 << 26) // ((q_heads + k_heads) * head)),
                    q_heads=q_heads, k_heads=k_heads, head_dim=head, rotary_dim=rng.choice([head, head, head // 2]),
                    max_position=_log(rng, 1024, 131072), layout=rng.choice(["interleaved", "half"]),
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), weight=rng.choice(["none", "same", "fp32"]),
                    table=rng.choice(["bf16", "fp32"]))
    if op == "pack":
        heads, layers = rng.choice([1, 2, 8, 16]), rng.randint(1, 6)
        return dict(op=op, layers=layers, tokens=_log(rng, 1, (1 << 18) // (heads * layers)), heads=heads,
                    block_size=rng.choice([1, 16, 16, 24, 64]), skipped=rng.choice([0.0, 0.1]))
    heads, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 5, 8])
    batch, nodes, ctx = _log(rng, 1, 64), _log(rng, 1, 100), _log(rng, 1, 65536)
    window = _log(rng, 16, 8192) if op == "window" or rng.random() < 0.2 else 0
    if op == "window" and rng.random() < 0.3:
        nodes, batch = _log(rng, 100, 4096), rng.randint(1, 2)
    while batch * heads * ctx > 1 << 21 or batch * heads * group * nodes * (ctx + nodes) > 1 << 28:
        ctx = max(1, ctx // 2 + rng.randint(0, 1))
        batch, nodes = max(1, batch - batch // 3), max(1, nodes - nodes // 8)
    return dict(op=op, batch=batch, heads=heads, group=group, nodes=nodes, max_ctx=ctx,
                block_size=rng.choice([8, 16, 16, 24, 64]), tree=nodes <= 100 and rng.random() < 0.6,
                softcap=rng.choice([0.0, 0.0, 30.0]), window=window, sinks=rng.choice([0, 4, 7]) if window else 0,
                lens_seed=rng.randrange(1 << 30))


def _lens(case):
    """The sequences' context lengths and drafted tokens: the first is the longest, the others ragged."""
    rng = random.Random(case["lens_seed"])
    ctx = [case["max_ctx"]] + [rng.randint(max(1, case["max_ctx"] // 4), case["max_ctx"])
                               for _ in range(case["batch"] - 1)]
    nodes = [case["nodes"]] + [rng.randint(max(1, case["nodes"] // 2), case["nodes"])
                               for _ in range(case["batch"] - 1)]
    return ctx, nodes


def _size(name):
    return 4 if name == "fp32" else 2


def _weight_type(case):
    return case["type"] if case["weight"] == "same" else case["weight"]


def work(case):
    if case["op"] == "prepare":
        heads, d = case["q_heads"] + case["k_heads"], case["head_dim"]
        n = case["tokens"] * heads * d
        rows = min(case["tokens"], case["max_position"])
        bytes_ = (3 if case["grad"] else 2) * n * _size(case["type"]) + 8 * case["tokens"]
        bytes_ += rows * case["rotary_dim"] * _size(case["table"])
        if case["weight"] != "none":
            bytes_ += (4 if case["grad"] else 2) * d * _size(_weight_type(case))
        turned = case["tokens"] * heads * case["rotary_dim"]
        return {"bytes": bytes_, "flops": (11 if case["grad"] else 4) * n + 3 * turned}
    if case["op"] == "pack":
        cells = case["layers"] * case["tokens"] * case["heads"]
        # rows in, cells out, cells in, rows out
        return {"bytes": cells * 2 * (4 * HEAD + 68) + 2 * 8 * case["tokens"], "flops": cells * 2 * HEAD * 4}
    ctx, nodes = _lens(case)
    H, G, W, S = case["heads"], case["group"], case["window"], case["sinks"]
    cell = 68 if case["op"] == "fp4" else 4 * HEAD
    keys = rows = pairs = 0
    for c, n in zip(ctx, nodes):
        rows += n * H * G
        if not W:
            keys += c + n
            pairs += n * c + (n * n if case["tree"] else n * (n + 1) // 2)
        else:
            keys += min(c + n, S + W + n - 1)
            # a tree's rows stand at different depths; counted as a chain's
            pairs += sum(min(c + i + 1, W + min(S, max(0, c + i + 1 - W))) for i in range(n))
    return {"bytes": keys * H * cell + rows * (4 * HEAD + 4), "flops": 4 * HEAD * pairs * H * G}


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


def _page_bytes(block_size):
    return (68 * block_size + 15) // 16 * 16


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t.normal_(0.0, scale, generator=gen)

    if case["op"] == "prepare":
        R, d, T = case["rotary_dim"], case["head_dim"], case["tokens"]
        half = R // 2
        f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        angle = torch.arange(case["max_position"], dtype=torch.float64, device=dev)[:, None] * f
        s = dict(case, cos_sin=torch.cat([angle.cos(), angle.sin()], dim=1).to(TYPES[case["table"]]), eps=1e-6,
                 positions=torch.randint(0, case["max_position"], (T,), generator=gen, device=dev))
        for part, heads in (("q", case["q_heads"]), ("k", case["k_heads"])):
            s[part] = normal(T, heads, d, scale=1.5, dtype=TYPES[case["type"]])
            s["grad_" + part] = normal(T, heads, d, dtype=TYPES[case["type"]]) if case["grad"] else None
            s[part + "_weight"] = None
            if case["weight"] != "none":
                w = 1.0 + 0.2 * normal(d, dtype=torch.float32)
                s[part + "_weight"] = w.to(TYPES[_weight_type(case)])
        return s
    if case["op"] == "pack":
        L, T, H, bs = case["layers"], case["tokens"], case["heads"], case["block_size"]
        blocks = (T + bs - 1) // bs + 4
        slots = torch.randperm(blocks * bs, generator=host)[:T]
        slots[torch.rand(T, generator=host) < case["skipped"]] = -1
        # as the projection leaves them: K's heads, then V's, in one row; K's channels of different sizes
        kv = normal(L, T, 2, H, HEAD)
        kv[:, :, 0] *= torch.exp(0.5 * normal(H, HEAD, dtype=torch.float32)).to(torch.bfloat16)
        return dict(case, k=kv[:, :, 0], v=kv[:, :, 1], slots=slots.to(dev),
                    caches=torch.zeros(L, blocks, H, _page_bytes(bs), dtype=torch.uint8, device=dev))

    lens, nodes = _lens(case)
    H, G, bs, T = case["heads"], case["group"], case["block_size"], sum(nodes)
    tables, blocks = _pages([c + n for c, n in zip(lens, nodes)], bs, host)
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    cache = normal(blocks, H, bs, 2 * HEAD)
    if case["op"] == "fp4":
        packed = torch.zeros(blocks, H, _page_bytes(bs), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 25) // (H * bs * 2 * HEAD))
        for b in range(0, blocks, step):
            codes, exps = _quantize(cache[b:b + step].unflatten(-1, (4, 32)))
            _put(packed[b:b + step], codes, exps, bs)
        cache = packed
    return dict(case, q=normal(T, H * G, HEAD, scale=2.0), cache=cache, tables=tables.to(dev),
                ctx_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                q_starts=torch.tensor(starts, dtype=torch.int32, device=dev),
                tree_mask=_tree_words(case, nodes, rng).to(dev) if case["tree"] else None)


# ---- norms and rotation -------------------------------------------------------------------------------------------

def _pairs(x, R, layout):
    return (x[..., 0:R:2], x[..., 1:R:2]) if layout == "interleaved" else (x[..., :R // 2], x[..., R // 2:R])


def _turn(x, s, sign):
    """x [T, H, d] in 32 bits with its first R elements turned (sign -1: back)."""
    R = s["rotary_dim"]
    row = s["cos_sin"][s["positions"]].float()[:, None, :]
    c, n = row[..., :R // 2], row[..., R // 2:] * sign
    a, b = _pairs(x, R, s["layout"])
    first, second = a * c - b * n, b * c + a * n
    turned = (torch.stack([first, second], dim=-1).flatten(-2) if s["layout"] == "interleaved"
              else torch.cat([first, second], dim=-1))
    return torch.cat([turned, x[..., R:]], dim=-1)


def _prepare(s):
    out, grads = [], []
    for part in ("q", "k"):
        x, w = s[part].float(), s[part + "_weight"]
        unit = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"])
        if not s["grad"]:
            out.append(_turn(unit if w is None else unit * w.float(), s, 1.0).to(s[part].dtype))
            continue
        r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"])
        g = _turn(s["grad_" + part].float(), s, -1.0)
        if w is not None:
            grads.append((g * unit).flatten(0, 1).sum(dim=0, dtype=torch.float64).to(w.dtype))
            g = g * w.float()
        dx = r * (g - unit * (g * unit).mean(dim=-1, keepdim=True))
        out.append(dx.to(s[part].dtype))
    return tuple(out + grads)


# ---- cells of 4 bits ----------------------------------------------------------------------------------------------

_STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _quantize(x):
    """x [..., 32] -> (codes 0 .. 15, exponents [...]) of its groups."""
    x = x.float()
    most = x.abs().amax(dim=-1)
    fraction, e = torch.frexp(most)  # most = fraction 2^e, fraction in [1/2, 1): at most 6 2^(e - 3) up to 3/4
    e = torch.where(fraction > 0.75, e - 2, e - 3)
    e = torch.where(most > 0, e, torch.full_like(e, -120)).clamp(-120, 125)
    y = torch.ldexp(x, -e[..., None])
    # nearest, ties to the even code: the middles belong to the lower code where that is even
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i in range(7):
        middle = (_STEPS[i] + _STEPS[i + 1]) / 2
        code += a > middle if i % 2 == 0 else a >= middle
    return code | (torch.signbit(x).to(torch.uint8) << 3), e


def _values(codes, exps):
    """What codes [..., 32] and exponents [...] stand for, in 32 bits."""
    steps = torch.tensor(_STEPS + [-v for v in _STEPS], device=codes.device)
    return torch.ldexp(steps[codes.long()], exps[..., None])


def _put(cache, codes, exps, bs):
    """All cells of pages: codes [blocks, H, bs, 4, 32], exponents [blocks, H, bs, 4] into cache [blocks, H, page]."""
    two = codes[..., 0::2] | codes[..., 1::2] << 4
    cache[..., :32 * bs] = two[..., :2, :].flatten(2)
    cache[..., 32 * bs:64 * bs] = two[..., 2:, :].flatten(2)
    cache[..., 64 * bs:68 * bs] = (exps + 127).to(torch.uint8).flatten(2)


def _cells(cache, block, page, bs):
    """K and V [..., H, 64] in 32 bits of the cells at (block, page), index tensors of one shape."""
    def run(first, width):
        at = first + page[..., None] * width + torch.arange(width, device=cache.device)
        # [..., width, H]: an index before and one behind the slice put the indexed axes in front
        return cache[block[..., None], :, at].transpose(-1, -2)

    exps = run(64 * bs, 4).int() - 127
    halves = []
    for part in range(2):
        two = run(32 * bs * part, 32)
        codes = torch.stack([two & 15, two >> 4], dim=-1).flatten(-2).unflatten(-1, (2, 32))
        halves.append(_values(codes, exps[..., 2 * part:2 * part + 2]).flatten(-2))
    return halves


def _pack(s):
    """The rows into their slots' cells, then those cells' values."""
    L, bs, H = s["layers"], s["block_size"], s["heads"]
    there = s["slots"] >= 0
    slot = s["slots"][there]
    block, page = slot // bs, slot % bs
    ks, vs = [], []
    for l in range(L):
        rows = torch.cat([s["k"][l][there], s["v"][l][there]], dim=-1).unflatten(-1, (4, 32))
        codes, exps = _quantize(rows)  # [rows, H, 4, 32], [rows, H, 4]
        two = codes[..., 0::2] | codes[..., 1::2] << 4
        for part in range(2):
            at = 32 * bs * part + page[:, None] * 32 + torch.arange(32, device=slot.device)
            s["caches"][l][block[:, None], :, at] = two[:, :, 2 * part:2 * part + 2].flatten(2).transpose(1, 2)
        at = 64 * bs + page[:, None] * 4 + torch.arange(4, device=slot.device)
        s["caches"][l][block[:, None], :, at] = (exps + 127).to(torch.uint8).transpose(1, 2)
        for out, part in zip((ks, vs), _cells(s["caches"][l], block, page, bs)):
            whole = torch.zeros(s["tokens"], H, HEAD, dtype=torch.bfloat16, device=slot.device)
            whole[there] = part.to(torch.bfloat16)
            out.append(whole)
    return torch.stack(ks), torch.stack(vs)


# ---- attention ----------------------------------------------------------------------------------------------------

def _attend(s):
    """All sequences' rows, a slice of the batch and of the nodes at a time."""
    T, heads = s["q"].shape[:2]
    H, G, W, S, bs, dev = s["heads"], s["group"], s["window"], s["sinks"], s["block_size"], s["q"].device
    out = torch.empty(T + 1, heads, HEAD, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(T + 1, heads, dtype=torch.float32, device=dev)
    starts, ctx_all = s["q_starts"].long(), s["ctx_lens"].long()
    # nodes at a time: few enough that a window's keys are not mostly other rows'
    step = s["nodes"] if s["tree"] or s["nodes"] <= 128 else 128
    for n0 in range(0, s["nodes"], step):
        n = min(step, s["nodes"] - n0)
        width = s["max_ctx"] + s["nodes"] if not W else min(s["max_ctx"] + s["nodes"], S + W + (s["nodes"] if s["tree"] else n))
        each = max(1, (1 << 28) // (heads * n * width))
        for b0 in range(0, s["batch"], each):
            seq = slice(b0, min(b0 + each, s["batch"]))
            first, count, ctx = starts[:-1][seq], (starts[1:] - starts[:-1])[seq], ctx_all[seq]
            node = n0 + torch.arange(n, device=dev)
            live = node < count[:, None]
            rows = (first[:, None] + node).clamp(max=T - 1)
            # the keys that any of these rows sees: the sinks, then all from the first one's window on
            key = torch.arange(width, device=dev).expand(ctx.shape[0], -1)
            if W:
                begin = (ctx + (0 if s["tree"] else n0) - W + 1).clamp(min=S)
                key = torch.where(key < S, key, key - S + begin[:, None])
            block = (key // bs).clamp(max=s["tables"].shape[1] - 1)
            page = torch.gather(s["tables"][seq].long(), 1, block)
            if s["op"] == "fp4":
                k, v = (t.transpose(1, 2) for t in _cells(s["cache"], page, key % bs, bs))  # [b, H, keys, 64]
            else:
                cell = s["cache"][page, :, key % bs].float().transpose(1, 2)
                k, v = cell[..., :HEAD], cell[..., HEAD:]
            q = s["q"][rows].float().view(-1, n, H, G, HEAD).permute(0, 2, 1, 3, 4).reshape(-1, H, n * G, HEAD)
            score = torch.matmul(q, k.transpose(2, 3).contiguous()).view(-1, H, n, G, width) * 0.125
            if s["softcap"]:
                score = s["softcap"] * torch.tanh(score / s["softcap"])
            other = key - ctx[:, None]  # the node that a key holds, negative for the context
            near = torch.ones_like(live)[:, :, None].expand(-1, -1, width)
            if s["tree"]:
                words = s["tree_mask"][rows]  # [b, nodes, words]
                at = other.clamp(0, 64 * words.shape[2] - 1)[:, None, :].expand(-1, n, -1)
                bit = ((torch.gather(words, 2, at // 64) >> (at % 64)) & 1 == 1) & (other < count[:, None])[:, None, :]
                context = (other < 0)[:, None, :]
                if W:
                    depth = (bit & ~context).sum(dim=2)  # nodes seen, the row's own among them
                    near = (key < S)[:, None, :] | (other[:, None, :] > (depth - 1 - W)[:, :, None])
                sees = torch.where(context, near, bit)
            else:
                if W:
                    near = (key < S)[:, None, :] | (other[:, None, :] > (node - W)[None, :, None])
                sees = (other[:, None, :] <= node[None, :, None]) & near
            sees = sees & live[:, :, None]
            score = score.masked_fill(~sees[:, None, :, None, :], -math.inf)
            top = score.amax(dim=-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            p = torch.exp(score - top)
            total = p.sum(dim=-1, keepdim=True)
            o = torch.matmul(p.view(-1, H, n * G, width), v.contiguous()).view(-1, H, n, G, HEAD)
            o = torch.where(total > 0, o / total, torch.zeros_like(o))
            # rows past a sequence's nodes go to a spare last row
            at = torch.where(live, rows, torch.full_like(rows, T)).flatten()
            out.index_copy_(0, at, o.transpose(1, 2).flatten(2, 3).flatten(0, 1).to(torch.bfloat16))
            lse.index_copy_(0, at, (top + torch.log(total)).squeeze(-1).transpose(1, 2).flatten(2, 3).flatten(0, 1))
    return out[:T], lse[:T]


# ---- one pass -----------------------------------------------------------------------------------------------------

def _own(s):
    import norm_rope_cache_amd as nrc

    if s["op"] == "prepare":
        if s["grad"]:
            dq, dk, dqw, dkw = nrc.qk_norm_rotate_grad(s["grad_q"], s["grad_k"], s["q"], s["k"], s["positions"],
                                                       s["cos_sin"], s["q_weight"], s["k_weight"], eps=s["eps"],
                                                       layout=s["layout"])
            return (dq, dk) if dqw is None else (dq, dk, dqw, dkw)
        return nrc.qk_norm_rotate(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_weight"], s["k_weight"],
                                  eps=s["eps"], layout=s["layout"])
    if s["op"] == "pack":
        nrc.context_fp4_store(s["k"], s["v"], s["slots"], s["caches"])
        return nrc.context_fp4_load(s["caches"], s["slots"])
    call = nrc.context_fp4_attention if s["op"] == "fp4" else nrc.context_window_attention
    return call(s["q"], s["cache"], s["tables"], s["ctx_lens"], s["q_starts"], s["nodes"], window=s["window"],
                sinks=s["sinks"], max_ctx=s["max_ctx"], tree_mask=s["tree_mask"], softcap=s["softcap"])


def run(state):
    if own:
        return _own(state)
    return {"prepare": _prepare, "pack": _pack, "fp4": _attend, "window": _attend}[state["op"]](state)


# ---- 64 bits ------------------------------------------------------------------------------------------------------

def _exact_prepare(s):
    """The definition in complex numbers, and its gradients by differentiation."""
    R, out, grads = s["rotary_dim"], [], []
    row = s["cos_sin"].double()[s["positions"]]
    turn = torch.complex(row[:, :R // 2].contiguous(), row[:, R // 2:].contiguous())[:, None, :]
    for part in ("q", "k"):
        x = s[part].double().requires_grad_(s["grad"])
        w = s[part + "_weight"]
        gain = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
        gain.requires_grad_(s["grad"])
        n = x / torch.sqrt(x.square().sum(dim=-1, keepdim=True) / x.shape[-1] + s["eps"]) * gain
        a, b = _pairs(n, R, s["layout"])
        z = torch.complex(a.contiguous(), b.contiguous()) * turn
        y = (torch.view_as_real(z).flatten(-2) if s["layout"] == "interleaved" else torch.cat([z.real, z.imag], dim=-1))
        y = torch.cat([y, n[..., R:]], dim=-1)
        if not s["grad"]:
            out.append(y)
            continue
        dx, dw = torch.autograd.grad(y, (x, gain), s["grad_" + part].double())
        out.append(dx)
        if w is not None:
            grads.append(dw)
    return tuple(out + grads)


def _exact_pack(s):
    """Every element by its distances to the codes' values, the group's exponent by trying."""
    steps = torch.tensor(_STEPS, dtype=torch.float64, device=s["slots"].device)
    there = (s["slots"] >= 0).double()[None, :, None, None]
    outs = []
    for rows in (s["k"], s["v"]):
        x = rows.double().unflatten(-1, (2, 32))
        most = x.abs().amax(dim=-1, keepdim=True)
        e = torch.floor(torch.log2(most.clamp(min=2.0 ** -140))) - 4
        for _ in range(4):
            e = torch.where(most > 6 * torch.exp2(e), e + 1, e)
        scale = torch.exp2(e.clamp(-120, 125))
        mags = (x.abs() / scale).unsqueeze(-1)
        code = torch.zeros(x.shape, dtype=torch.int64, device=x.device)
        best = torch.full(x.shape, math.inf, dtype=torch.float64, device=x.device)
        for i in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they keep ties
            far = (mags[..., 0] - steps[i]).abs()
            code, best = torch.where(far < best, i, code), torch.minimum(best, far)
        outs.append((steps[code] * scale * torch.sign(x)).flatten(-2) * there)
    return tuple(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prepare":
        return _exact_prepare(s)
    if case["op"] == "pack":
        return _exact_pack(s)
    T, heads = s["q"].shape[:2]
    dev, H, G, bs, W, S = s["q"].device, s["heads"], s["group"], s["block_size"], s["window"], s["sinks"]
    lut = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device=dev) / 2
    out = torch.zeros(T, heads, HEAD, dtype=torch.float64, device=dev)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device=dev)
    for b in range(s["batch"]):
        lo, hi = (int(v) for v in s["q_starts"][b:b + 2])
        ctx, n = int(s["ctx_lens"][b]), hi - lo
        keys = ctx + n
        at = torch.arange(keys, device=dev)
        page = s["tables"][b].long()[at // bs]
        sees = np.ones((n, keys), dtype=bool)
        if s["tree_mask"] is None:
            sees[:, ctx:] = np.tril(np.ones((n, n), dtype=bool))
            where = ctx + np.arange(n)
        else:
            words = s["tree_mask"][lo:hi].cpu().numpy().view(np.uint8)
            sees[:, ctx:] = np.unpackbits(words, axis=1, bitorder="little")[:, :n].astype(bool)
            where = ctx + sees[:, ctx:].sum(axis=1) - 1
        if W:
            inside = (np.arange(keys)[None, :] < S) | (np.arange(keys)[None, :] + W > where[:, None])
            last = keys if s["tree_mask"] is None else ctx  # a tree's nodes are seen by the mask alone
            sees[:, :last] &= inside[:, :last]
        sees = torch.from_numpy(sees).to(dev)
        for h in range(H):
            if s["op"] == "fp4":
                pages = s["cache"][page, h].long()  # [keys, page bytes]
                scale = torch.exp2(torch.gather(pages, 1, 64 * bs + (at % bs * 4)[:, None] + torch.arange(4, device=dev)).double() - 127)
                kv = []
                for part in range(2):
                    byte = torch.gather(pages, 1, 32 * bs * part + (at % bs * 32)[:, None] + torch.arange(32, device=dev))
                    val = torch.empty(keys, HEAD, dtype=torch.float64, device=dev)
                    val[:, 0::2], val[:, 1::2] = lut[byte % 16], lut[byte // 16]
                    val[:, :32] *= scale[:, 2 * part:2 * part + 1]
                    val[:, 32:] *= scale[:, 2 * part + 1:2 * part + 2]
                    kv.append(val)
                k, v = kv
            else:
                cell = s["cache"][page, h, at % bs].double()
                k, v = cell[:, :HEAD], cell[:, HEAD:]
            step = max(1, (1 << 27) // (G * keys))
            for i in range(0, n, step):
                z = slice(i, min(i + step, n))
                q = s["q"][lo + z.start:lo + z.stop, h * G:(h + 1) * G].double()
                score = (q.reshape(-1, HEAD) @ k.T.contiguous()).reshape(-1, G, keys) / 8.0
                if s["softcap"]:
                    score = torch.tanh(score / s["softcap"]) * s["softcap"]
                score = score.masked_fill(~sees[z][:, None, :], -math.inf)
                l = torch.logsumexp(score, dim=-1)
                p = torch.exp(score - l[..., None])
                out[lo + z.start:lo + z.stop, h * G:(h + 1) * G] = (p.reshape(-1, keys) @ v).reshape(-1, G, HEAD)
                lse[lo + z.start:lo + z.stop, h * G:(h + 1) * G] = l
    return out, lse
