"""Attention over a key/value cache, as one decoder layer of the multi-variant server runs it: prefill and decode with a
sliding window and always visible first tokens, decode for requests that share prefixes, decode that accumulates
attention weights, and the eviction that those weights drive.

One cache of a layer is K, V [slots, capacity, kv_heads, head_dim] bf16; a request owns a slot.  With P keys of a shared
prefix (0 without) the position of prefix key j is j and that of own key j is P + j; a query at position t sees position p
if p <= t and (p < sinks or window == 0 or p > t - window).  A query that sees nothing gives zeros."""
import math

import torch

own = False

# ---------------------------------------------------------------------------------------------------------------------
# The cases.  64 query heads, 8 key/value heads, head_dim 128 and 128 requests a decode step over 14 variants are this
# repository's decoder-layer workload; the other head layouts are generic ones.
# ---------------------------------------------------------------------------------------------------------------------


def listed():
    wide = {"q_heads": 64, "kv_heads": 8, "head_dim": 128}
    return [
        # the smallest decode call: one user, a short chat; latency counts
        {"name": "decode_one", "op": "decode", "batch": 1, "shortest": 300, "longest": 300, "window": 0, "sinks": 0, **wide},
        # the stack's decode batch with ragged lengths and a windowed layer
        {"name": "decode_window", "op": "decode", "batch": 128, "shortest": 1, "longest": 16384, "window": 4096, "sinks": 4, **wide},
        # a few very long documents, everything visible
        {"name": "decode_long", "op": "decode", "batch": 4, "shortest": 90001, "longest": 131072, "window": 0, "sinks": 0, **wide},
        # a few short prompts that start a chat, odd lengths, one of a single token
        {"name": "prefill_short", "op": "prefill", "batch": 3, "shortest": 1, "longest": 131, "before": 0, "window": 0, "sinks": 0, **wide},
        # ragged prompts of a windowed layer, the later chunks of longer ones
        {"name": "prefill_window", "op": "prefill", "batch": 8, "shortest": 333, "longest": 2048, "before": 700, "window": 1024, "sinks": 4, **wide},
        # one long prompt, everything visible: the largest call
        {"name": "prefill_long", "op": "prefill", "batch": 1, "shortest": 8192, "longest": 8192, "before": 0, "window": 0, "sinks": 0, **wide},
        # one long system prompt that a whole batch shares, short own parts
        {"name": "prefix_one", "op": "prefix", "batch": 64, "shortest": 1, "longest": 1024, "prefixes": 1, "prefix_short": 16384, "prefix_long": 16384,
         "window": 0, "sinks": 0, **wide},
        # the stack's decode batch: every variant has a prompt of its own, requests spread over the variants by Zipf's law
        {"name": "prefix_variants", "op": "prefix", "batch": 128, "shortest": 1, "longest": 700, "prefixes": 14, "prefix_short": 500, "prefix_long": 4096,
         "window": 0, "sinks": 0, **wide},
        # a small call that keeps count of where the attention went
        {"name": "weigh_small", "op": "weigh", "batch": 2, "shortest": 391, "longest": 777, "window": 0, "sinks": 0, "q_heads": 32, "kv_heads": 8, "head_dim": 64},
        # an ordinary decode step of a layer whose cache is kept to a budget
        {"name": "weigh_batch", "op": "weigh", "batch": 32, "shortest": 2049, "longest": 4608, "window": 0, "sinks": 0, **wide},
        # one request over a small odd budget
        {"name": "evict_one", "op": "evict", "batch": 1, "shortest": 1001, "longest": 1001, "budget": 700, "sinks": 4, "recent": 129, "q_heads": 32, "kv_heads": 8, "head_dim": 64},
        # a batch of requests that reached the end of their slots at about the same time
        {"name": "evict_batch", "op": "evict", "batch": 32, "shortest": 4100, "longest": 4608, "budget": 4096, "sinks": 4, "recent": 1024, **wide},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    q_heads, kv_heads, head_dim = rng.choice([(64, 8, 128), (64, 8, 128), (32, 8, 128), (32, 8, 64), (16, 16, 64), (48, 4, 128), (20, 4, 128), (16, 1, 128)])
    case = {"op": rng.choice(["decode", "decode", "prefill", "prefill", "prefix", "prefix", "weigh", "evict"]), "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim}
    window, sinks = rng.choice([(0, 0), (log(16, 4096), rng.choice([0, 1, 4, 64]))])
    if case["op"] == "decode":
        batch = log(1, 128)
        longest = log(1, min(131072, 128 * 16384 // batch))
        return {**case, "batch": batch, "shortest": log(1, longest), "longest": longest, "window": window, "sinks": sinks}
    if case["op"] == "prefill":
        batch = log(1, 16)
        longest = log(1, 4096 if batch < 3 else 1024)
        return {**case, "batch": batch, "shortest": log(1, longest), "longest": longest, "before": rng.choice([0, log(1, 2000)]), "window": window, "sinks": sinks}
    if case["op"] == "prefix":
        batch, prefix = log(2, 128), log(100, 8192)
        longest = log(1, 1024)
        return {**case, "batch": batch, "shortest": log(1, longest), "longest": longest, "prefixes": rng.choice([1, log(1, 14)]), "prefix_short": log(64, prefix),
                "prefix_long": prefix, "window": window, "sinks": sinks}
    if case["op"] == "weigh":
        longest = log(16, 4608)
        return {**case, "batch": log(1, 32), "shortest": log(1, longest), "longest": longest, "window": window, "sinks": sinks}
    longest = log(64, 4608)
    budget = rng.randint(longest // 2, longest)
    return {**case, "batch": log(1, 32), "shortest": log(longest // 4, longest), "longest": longest, "budget": budget, "sinks": min(4, budget // 4), "recent": log(1, budget // 2)}


def spread(lo, hi, n):
    """n lengths from lo to hi, the longest first."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def requests_of(case):
    """How many requests name each prefix: Zipf's law."""
    share = [1.0 / (k + 1) for k in range(case["prefixes"])]
    return [round(case["batch"] * x / sum(share)) for x in share]


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    hq, hk, d, n = case["q_heads"], case["kv_heads"], case["head_dim"], case["batch"]
    op = case["op"]
    new = spread(case["shortest"], case["longest"], n)
    own_max = case["longest"] + case.get("before", 0)
    prefixes = case.get("prefixes", 0)
    slots = 2 * n if op == "evict" else n + prefixes
    capacity = -(-max(own_max, case.get("prefix_long", 0)) // 16) * 16

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def shuffled(values):
        return whole(values)[torch.randperm(len(values), generator=g, device="cuda")]

    s = {"case": case, "scale": d ** -0.5}
    s["k"], s["v"] = normal(slots, capacity, hk, d), normal(slots, capacity, hk, d)
    order = torch.randperm(n, generator=g, device="cuda")
    if op == "evict":
        # the weight that a key has gathered over many steps: a few heavy keys, many light ones
        s["weights"] = torch.rand(slots, hk, capacity, generator=g, device="cuda").pow(8) * 50
        s["src"], s["dst"] = order.to(torch.int32), (n + torch.randperm(n, generator=g, device="cuda")).to(torch.int32)
        s["lens"] = torch.zeros(slots, dtype=torch.int32, device="cuda")
        s["lens"][:n] = shuffled(new)
        s["k"][n:], s["v"][n:], s["weights"][n:] = 0, 0, 0
        s["kept"] = torch.full((n, hk, case["budget"]), -1, dtype=torch.int32, device="cuda")
    else:
        s["slots"] = order.to(torch.int32)
        news = shuffled(new)
        tokens = sum(new) if op == "prefill" else n
        s["q"] = normal(tokens, hq, d) * 1.5
        s["out"] = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
        if op == "prefill":
            # how much of a request is in the cache before this chunk differs from request to request
            before = whole([case["before"] * i // max(1, n - 1) for i in range(n)])
            s["cu_q"] = torch.cat([whole([0]), news.cumsum(0, dtype=torch.int32)])
            s["lens"], s["longest_new"] = before + news, case["longest"]
        else:
            s["lens"] = news
        if op == "prefix":
            ids = [k for k, c in enumerate(requests_of(case)) for _ in range(c)]
            s["prefix_ids"] = shuffled((ids + [0] * n)[:n])
            s["prefix_slots"] = whole(list(range(n, n + prefixes)))
            s["prefix_lens"] = shuffled(spread(case["prefix_short"], case["prefix_long"], prefixes))
        if op == "weigh":
            s["weights"] = torch.rand(slots, hk, capacity, generator=g, device="cuda") * 0.01
    if own:
        import bit_delta_compressed_gb300 as bd

        s["bd"] = bd
        if op == "evict":
            s["workspace"] = bd.evict_workspace(n, hk, capacity, device="cuda")
        else:
            s["workspace"] = bd.attn_workspace(s["q"].shape[0], n, hq, hk, d, weigh_len=capacity if op == "weigh" else 0, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------------------------
# The plain form and the framework's calls
# ---------------------------------------------------------------------------------------------------------------------


def softmax_product(q, k, v, mask, scale):
    """Softmax over the masked last axis and the product with the values: q [.., r, d], k and v [.., n, d], mask [.., r, n]; 32 bits.
    The weights too; rows that see nothing are zero."""
    s = (q @ k.transpose(-1, -2)).mul_(scale)
    s.masked_fill_(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top.masked_fill_(top == -math.inf, 0.0)).exp_()
    p.div_(p.sum(-1, keepdim=True).clamp_min_(1e-30))
    return p @ v, p


def sees(at, pos, window, sinks):
    """Whether a query at position `at` sees position `pos`."""
    seen = pos <= at
    return seen & ((pos < sinks) | (pos > at - window)) if window else seen


def rows_of(cache, slots, longest):
    """The first keys of some slots, [n, kv_heads, longest, head_dim] in 32 bits; what lies behind the lengths is masked later."""
    return cache[slots.long(), :longest].float().transpose(1, 2)


def plain_prefill(s, c):
    k, v, n = s["k"], s["v"], c["batch"]
    group, hk = c["q_heads"] // c["kv_heads"], c["kv_heads"]
    token = torch.arange(s["q"].shape[0], device="cuda")
    of = torch.searchsorted(s["cu_q"][1:].contiguous(), token.to(torch.int32), right=True)
    i = token - s["cu_q"].long()[of]
    longest, keys = s["longest_new"], k.shape[1]
    q = torch.zeros(n, longest, c["q_heads"], c["head_dim"], device="cuda")
    q[of, i] = s["q"].float()
    q = q.view(n, longest, hk, group, -1).permute(0, 2, 3, 1, 4)
    news = s["cu_q"][1:] - s["cu_q"][:-1]
    at = (s["lens"] - news)[:, None] + torch.arange(longest, device="cuda")
    pos = torch.arange(keys, device="cuda")
    mask = sees(at[:, None, None, :, None], pos, c["window"], c["sinks"])
    o, _ = softmax_product(q, rows_of(k, s["slots"], keys)[:, :, None], rows_of(v, s["slots"], keys)[:, :, None], mask, s["scale"])
    return o.permute(0, 3, 1, 2, 4).reshape(n, longest, c["q_heads"], c["head_dim"])[of, i].to(torch.bfloat16)


def plain_decode(s, c):
    k, v, n, longest = s["k"], s["v"], c["batch"], c["longest"]
    hk, group = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    keys, values = rows_of(k, s["slots"], longest), rows_of(v, s["slots"], longest)
    pos, lens = torch.arange(longest, device="cuda"), s["lens"][:, None]
    at = lens - 1
    valid = pos < lens
    if "prefix_ids" in s:
        of = s["prefix_ids"].long()
        p = s["prefix_lens"][of][:, None]
        front, most = torch.arange(c["prefix_long"], device="cuda"), c["prefix_long"]
        keys = torch.cat([rows_of(k, s["prefix_slots"][of], most), keys], 2)
        values = torch.cat([rows_of(v, s["prefix_slots"][of], most), values], 2)
        valid = torch.cat([front < p, valid], 1)
        pos, at = torch.cat([front.expand(n, -1), p + pos], 1), at + p
    mask = valid & sees(at, pos, c["window"], c["sinks"])
    q = s["q"].float().view(n, hk, group, -1)
    o, weight = softmax_product(q, keys, values, mask[:, None, None], s["scale"])
    if "weights" in s:
        s["weights"][s["slots"].long(), :, :longest] += weight.sum(2)
    return o.reshape(n, c["q_heads"], c["head_dim"]).to(torch.bfloat16)


def plain_evict(s, c):
    src, dst, budget = s["src"].long(), s["dst"].long(), c["budget"]
    n, lens = src.numel(), s["lens"][src.long()]
    w = s["weights"][src][:, :, : c["longest"]]
    pos = torch.arange(c["longest"], device="cuda")
    valid = pos < lens[:, None]
    stays = (pos < c["sinks"]) | (pos >= lens[:, None] - c["recent"])
    rank = torch.where(valid[:, None], torch.where(stays[:, None], math.inf, w), -math.inf)
    heaviest = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = lens.clamp_max(budget)
    column = torch.arange(budget, device="cuda")
    kept = torch.where(column < keep[:, None, None], heaviest, c["longest"]).sort(-1).values
    valid = (column < keep[:, None])[:, None].expand(kept.shape)
    at = kept.clamp_max(c["longest"] - 1)
    head = torch.arange(c["kv_heads"], device="cuda")[None, :, None]
    b, h, j = valid.nonzero(as_tuple=True)
    for_row = (src[b], at[b, h, j], h)
    to_row = (dst[b], j, h)
    s["k"][to_row], s["v"][to_row] = s["k"][for_row], s["v"][for_row]
    s["weights"][dst[b], h, j] = s["weights"][src[:, None, None].expand(n, head.numel(), budget)[valid], h, at[valid]]
    s["lens"][dst] = keep
    s["kept"].copy_(torch.where(valid, kept, -1))


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if op == "evict":
        if own:
            s["bd"].cache_evict(s["k"], s["v"], s["weights"], s["lens"], s["src"], s["dst"], c["budget"], s["workspace"], sinks=c["sinks"], recent=c["recent"],
                                kept=s["kept"])
        else:
            plain_evict(s, c)
        n = c["batch"]
        return {"k": s["k"][n:], "v": s["v"][n:], "weights": s["weights"][n:], "lens": s["lens"][n:], "kept": s["kept"]}
    if own:
        mask = {"window": c["window"], "sinks": c["sinks"], "scale": s["scale"], "slots": s["slots"], "out": s["out"]}
        if op == "prefill":
            s["bd"].attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["lens"], s["workspace"], **mask)
        elif op == "prefix":
            s["bd"].attn_decode_prefix(s["q"], s["k"], s["v"], s["lens"], s["prefix_ids"], s["prefix_slots"], s["prefix_lens"], s["workspace"], **mask)
        elif op == "weigh":
            s["bd"].attn_decode(s["q"], s["k"], s["v"], s["lens"], s["workspace"], weights=s["weights"], **mask)
            return {"out": s["out"], "weights": s["weights"]}
        else:
            s["bd"].attn_decode(s["q"], s["k"], s["v"], s["lens"], s["workspace"], **mask)
        return s["out"]
    o = plain_prefill(s, c) if op == "prefill" else plain_decode(s, c)
    return {"out": o, "weights": s["weights"]} if op == "weigh" else o


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------------------------------------


def work(case):
    hq, hk, d, n = case["q_heads"], case["kv_heads"], case["head_dim"], case["batch"]
    lengths = spread(case["shortest"], case["longest"], n)
    window, sinks = case.get("window", 0), case["sinks"]
    row = hk * d * 4  # one key and its value, all heads

    def visible(t):  # positions that a query at position t sees
        return t + 1 if not window else min(t + 1, window + min(sinks, max(0, t + 1 - window)))

    if case["op"] == "evict":
        kept = sum(min(x, case["budget"]) for x in lengths)
        return {"bytes": hk * (4 * sum(lengths) + kept * (8 * d + 4) + 4 * n * case["budget"]) + 8 * n, "flops": 0}
    if case["op"] == "prefill":
        pairs = keys = 0
        # which length meets which part before it differs by the seed: taken here in the order of prepare's own list
        for i, x in enumerate(lengths):
            before = case["before"] * i // max(1, n - 1)
            pairs += sum(visible(t) for t in range(before, before + x))
            keys += min(before + x, x - 1 + visible(before))
        return {"bytes": keys * row + 4 * sum(lengths) * hq * d, "flops": 4 * d * hq * pairs}
    if case["op"] == "prefix":
        p = spread(case["prefix_short"], case["prefix_long"], case["prefixes"])
        mean = sum(p) // len(p)
        seen = [visible(mean + x - 1) for x in lengths]
        mine = [min(x, window) if window else x for x in lengths]
        shared = sum(min(x, max(0, window + sinks - min(lengths))) if window else x for x in p)
        return {"bytes": (sum(mine) + shared) * row + 4 * n * hq * d, "flops": 4 * d * hq * sum(seen)}
    keys = sum(visible(x - 1) for x in lengths)
    return {"bytes": keys * (row + (8 * hk if case["op"] == "weigh" else 0)) + 4 * n * hq * d, "flops": 4 * d * hq * keys}


def exact(case, seed):
    s = prepare(case, seed)
    n, hq, hk = case["batch"], case["q_heads"], case["kv_heads"]
    lens = s["lens"].tolist()
    if case["op"] == "evict":
        result = {x: s[x][n:].clone() for x in ("weights", "k", "v")}
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            size, c = lens[a], min(lens[a], case["budget"])
            for h in range(hk):
                order = sorted(range(size), key=lambda j, w=s["weights"][a, h, :size].tolist(): (j >= case["sinks"] and j < size - case["recent"], -w[j], j))
                kept = torch.tensor(sorted(order[:c]), dtype=torch.long, device="cuda")
                result["k"][b - n, :c, h], result["v"][b - n, :c, h] = s["k"][a, kept, h], s["v"][a, kept, h]
                result["weights"][b - n, h, :c] = s["weights"][a, h, kept]
        return {"lens": None, "kept": None, **{x: t.double() for x, t in result.items()}}
    ends = s["cu_q"].tolist() if case["op"] == "prefill" else list(range(n + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if "weights" in s else None
    for b, slot in enumerate(s["slots"].tolist()):
        m, size = ends[b + 1] - ends[b], lens[b]
        front = int(s["prefix_lens"][s["prefix_ids"][b]]) if "prefix_ids" in s else 0
        at = torch.arange(front + size - m, front + size, device="cuda")[:, None]
        pos = torch.arange(front + size, device="cuda")
        hidden = pos > at
        if case["window"]:
            hidden = hidden | ((pos <= at - case["window"]) & (pos >= case["sinks"]))
        for h in range(hk):
            keys, values = s["k"][slot, :size, h].double(), s["v"][slot, :size, h].double()
            if front:
                shared = int(s["prefix_slots"][s["prefix_ids"][b]])
                keys, values = torch.cat([s["k"][shared, :front, h].double(), keys]), torch.cat([s["v"][shared, :front, h].double(), values])
            for j in range(h * hq // hk, (h + 1) * hq // hk):
                score = s["q"][ends[b]:ends[b + 1], j].double() @ keys.T * s["scale"]
                score = score.masked_fill_(hidden, -math.inf)
                p = torch.softmax(score, -1)
                out[ends[b]:ends[b + 1], j] = p @ values
                if weights is not None:
                    weights[slot, h, :size] += p[0, front:]
    return out if weights is None else {"out": out, "weights": weights}
