"""The operators around the MoE layer in a speculative decode step, as cases to measure.

A serving step with drafted tokens projects its hidden rows with 4-bit weights, turns queries and keys by
their positions and appends keys and values to a paged cache, lets every drafted token attend to the cache and
to its own ancestors in the draft tree, and at the end verifies the drafted tokens against the target's
probabilities.  `run` computes one of these in elementary torch operations, or, where `own` is true, through
the package's public calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of 32 drafted tokens: all of the head, halves layout, a context stretched by 4, keys
        # and values appended to the paged cache in the same call.
        {"name": "rope_step", "op": "rope", "dtype": "bf16", "tokens": 32, "q_heads": 32, "k_heads": 8, "dim": 128,
         "rot": 128, "offset": 0, "interleaved": False, "inverse": False, "base": 1.0e6, "factor": 4.0,
         "original": 32768, "far": 131072, "page": 16},
        # A long prompt: interleaved pairs in half of every head, positions up to a million.
        {"name": "rope_prompt", "op": "rope", "dtype": "bf16", "tokens": 16384, "q_heads": 64, "k_heads": 8,
         "dim": 128, "rot": 64, "offset": 0, "interleaved": True, "inverse": False, "base": 1.0e4, "factor": 40.0,
         "original": 4096, "far": 1000000, "page": 0},
        # Odd sizes: the last 64 of 192 wide heads (a positional part beside a plain one), one shared key head,
        # turned back (the gradient's direction, or a cached key that moves).
        {"name": "rope_back", "op": "rope", "dtype": "fp16", "tokens": 1001, "q_heads": 7, "k_heads": 1, "dim": 192,
         "rot": 64, "offset": 128, "interleaved": False, "inverse": True, "base": 1.0e4, "factor": 1.0,
         "original": 4096, "far": 32768, "page": 0},
        # One token through a square projection: a matrix-vector product in earnest.
        {"name": "linear_one", "op": "linear", "dtype": "bf16", "rows": 1, "inner": 7168, "outer": 7168, "group": 128,
         "gated": False},
        # The gate and up projections of a shared expert with SiLU and the product, four tokens.
        {"name": "linear_gated", "op": "linear", "dtype": "bf16", "rows": 4, "inner": 7168, "outer": 2048, "group": 128,
         "gated": True},
        # The output head over a whole vocabulary for eight drafted tokens.
        {"name": "linear_vocab", "op": "linear", "dtype": "bf16", "rows": 8, "inner": 7168, "outer": 129280,
         "group": 128, "gated": False},
        # Ragged: thirteen rows, odd output width, an inner size that ends inside a block, small groups.
        {"name": "linear_ragged", "op": "linear", "dtype": "fp16", "rows": 13, "inner": 4000, "outer": 11003,
         "group": 32, "gated": False},
        # The first step of one short conversation: latency.
        {"name": "tree_first", "op": "tree", "dtype": "bf16", "batch": 1, "nodes": 5, "chain": False, "q_heads": 32,
         "k_heads": 8, "dim": 128, "page": 16, "shortest": 37, "longest": 37, "heads_first": False},
        # A batch of ordinary requests with short chains of drafted tokens.
        {"name": "tree_batch", "op": "tree", "dtype": "bf16", "batch": 32, "nodes": 4, "chain": True, "q_heads": 32,
         "k_heads": 8, "dim": 128, "page": 16, "shortest": 300, "longest": 4100, "heads_first": False},
        # Two very long documents with the widest tree.
        {"name": "tree_long", "op": "tree", "dtype": "bf16", "batch": 2, "nodes": 64, "chain": False, "q_heads": 64,
         "k_heads": 4, "dim": 128, "page": 64, "shortest": 100003, "longest": 131072, "heads_first": False},
        # Chains of seven drafted tokens for 32 requests, with the draft model's probabilities.
        {"name": "verify_chain", "op": "verify", "batch": 32, "nodes": 7, "chain": True, "vocab": 129280},
        # Trees of 24 candidates for two requests, a vocabulary of odd size.
        {"name": "verify_tree", "op": "verify", "batch": 2, "nodes": 24, "chain": False, "vocab": 32003},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "linear", "tree", "tree", "verify"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, 32])
        k_heads = rng.choice([1, 2, 4, 8, 16])
        page = rng.choice([0, 16, 24, 64])
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "tokens": _log(rng, 1, 2048 if page else 16384), "q_heads": k_heads * rng.choice([1, 2, 4, 7]),
                "k_heads": k_heads, "dim": dim, "rot": rot, "offset": rng.choice([0, (dim - rot) // 8 * 8]),
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.25,
                "base": rng.choice([1.0e4, 5.0e5, 1.0e6]), "factor": rng.choice([1.0, 1.0, 4.0, 40.0]),
                "original": rng.choice([4096, 32768]), "far": _log(rng, 100, 1000000), "page": page}
    if op == "linear":
        rows, inner = _log(rng, 1, 64), 32 * _log(rng, 4, 576)
        gated = rng.random() < 0.3
        outer = _log(rng, 1, min(131072, 463000000 // inner) // (2 if gated else 1))
        group = rng.choice([g for g in (32, 64, 128) if inner % g == 0])
        return {"op": op, "dtype": dtype, "rows": rows, "inner": inner, "outer": outer, "group": group, "gated": gated}
    if op == "tree":
        k_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        nodes = rng.choice([1, 1, 2, 4, 5, 8, 16, 24, 33, 64])
        longest = _log(rng, 1, 65536)
        batch = max(1, min(_log(rng, 1, 64), 262144 // (k_heads * longest)))
        return {"op": op, "dtype": dtype, "batch": batch, "nodes": nodes, "chain": rng.random() < 0.3,
                "q_heads": k_heads * group, "k_heads": k_heads, "dim": rng.choice([64, 128, 128]),
                "page": rng.choice([1, 16, 16, 32, 48, 64, 256]), "shortest": rng.randint(0, longest),
                "longest": longest, "heads_first": rng.random() < 0.3}
    return {"op": op, "batch": _log(rng, 1, 32), "nodes": _log(rng, 1, 31), "chain": rng.random() < 0.5,
            "vocab": _log(rng, 1000, 130000)}


def work(case):
    op = case["op"]
    if op == "rope":
        size = torch.finfo(TYPES[case["dtype"]]).bits // 8
        values = case["tokens"] * (case["q_heads"] + case["k_heads"]) * (case["dim"] if case["page"] else case["rot"])
        if case["page"]:
            values += case["tokens"] * case["k_heads"] * (case["dim"])
        return {"bytes": 2 * size * values + 4 * case["tokens"],
                "flops": 3 * case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["rot"]}
    if op == "linear":
        m, k, n = case["rows"], case["inner"], case["outer"]
        stored = n * (2 if case["gated"] else 1)
        return {"bytes": stored * k // 2 + stored * (k // case["group"]) * 4 + 2 * m * (k + n), "flops": 2 * m * k * stored}
    if op == "tree":
        lengths, counts = _tree_sizes(case)
        hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
        slots = sum(lengths) + sum(counts)
        return {"bytes": 4 * slots * hk * d + 4 * sum(counts) * hq * d,
                "flops": 4 * d * hq * sum(c * (n + c) for n, c in zip(lengths, counts))}
    b, n, v = case["batch"], case["nodes"], case["vocab"]
    return {"bytes": 4 * b * v * (2 if case["chain"] else 1) + 12 * b * n, "flops": 2 * b * v}


# ------------------------------------------------------------------------------------------------- inputs

def _frequencies(case):
    """Radians a position of every pair in 64 bits, and the factor on the result: plain, or stretched between the
    pairs that turn more than 32 times and those that turn less than once in the original context (YaRN)."""
    d, base, factor = case["rot"], case["base"], case["factor"]
    i = np.arange(d // 2, dtype=np.float64)
    f = base ** (-2.0 * i / d)
    if factor == 1.0:
        return f, 1.0
    low, high = (d * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0))
    low, high = max(math.floor(low), 0), min(math.ceil(high), d - 1)
    ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
    return f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0


def _tree_sizes(case):
    """Committed length and drafted tokens of every sequence."""
    r = np.random.default_rng([case["batch"], case["longest"], case["shortest"], case["nodes"]])
    lengths = r.integers(case["shortest"], case["longest"] + 1, case["batch"])
    lengths[0] = case["longest"]
    lengths[-1] = case["longest"] if case["batch"] == 1 else case["shortest"]
    counts = np.full(case["batch"], case["nodes"])
    if case["batch"] > 2:
        counts[1:-1] = r.integers(max(1, case["nodes"] // 2), case["nodes"] + 1, case["batch"] - 2)
    return [int(n) for n in lengths], [int(n) for n in counts]


def _parents(n, chain, r):
    """Parents of a draft tree's nodes, in an order that has a parent before its children; -1 is the root."""
    return np.arange(-1, n - 1) if chain else np.array([max(-1, int(r.integers(-1, j)) if r.random() < 0.5 else j // 2 - 1)
                                                       for j in range(n)])


def _ancestors(parents):
    """Bit masks of every node's ancestors and itself."""
    masks = []
    for j, p in enumerate(parents):
        masks.append((1 << j) | (masks[p] if p >= 0 else 0))
    return masks


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    s = dict(case)
    op = case["op"]
    if op == "rope":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        dt = TYPES[case["dtype"]]
        # the projections' output as a decoder has it: the rows of q, k and v side by side
        s["qkv"] = torch.randn(t, hq + 2 * hk, d, generator=g, device="cuda").to(dt)
        s["positions"] = torch.from_numpy(r.integers(0, case["far"], t).astype(np.int32)).cuda()
        f, s["scale"] = _frequencies(case)
        s["inv_freq"] = torch.from_numpy(f).cuda()
        if case["page"]:
            pages = -(-t // case["page"]) + 3
            s["k_cache"] = torch.zeros(pages, case["page"], hk, d, dtype=dt, device="cuda")
            s["v_cache"] = torch.zeros_like(s["k_cache"])
            slots = r.permutation(pages * case["page"])[:t].astype(np.int32)
            slots[r.random(t) < 0.1] = -1  # rows that only fill up a captured batch
            s["slots"] = torch.from_numpy(slots).cuda()
    elif op == "linear":
        m, k, n = case["rows"], case["inner"], case["outer"]
        stored = n * (2 if case["gated"] else 1)
        s["x"] = torch.randn(m, k, generator=g, device="cuda").to(TYPES[case["dtype"]])
        s["w"] = torch.randint(0, 256, (stored, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["w_scale"] = (0.5 + torch.rand(stored, k // case["group"], generator=g, device="cuda")) * (0.2 / math.sqrt(k))
    elif op == "tree":
        hq, hk, d, page = case["q_heads"], case["k_heads"], case["dim"], case["page"]
        lengths, counts = _tree_sizes(case)
        total, dt = sum(counts), TYPES[case["dtype"]]
        need = [-(-(n + c) // page) for n, c in zip(lengths, counts)]
        pool = sum(need) + 5
        shape = (pool, hk, page, d) if case["heads_first"] else (pool, page, hk, d)
        order = (0, 2, 1, 3) if case["heads_first"] else (0, 1, 2, 3)
        for name in ("k_cache", "v_cache"):
            s[name] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g).permute(order)
        s["q"] = torch.randn(total, hq, d, generator=g, device="cuda").to(dt)
        free = r.permutation(pool)
        table = np.full((len(need), max(need)), -1, dtype=np.int32)
        at = 0
        for b, p in enumerate(need):
            table[b, :p] = free[at:at + p]
            at += p
        s["block_table"] = torch.from_numpy(table).cuda()
        s["context_lens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        s["node_offsets"] = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
        masks = [m for c in counts for m in _ancestors(_parents(c, case["chain"], r))]
        s["tree_mask"] = torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64)).cuda()
        s["most"] = (max(n + c for n, c in zip(lengths, counts)), max(counts))
    else:
        b, n, v = case["batch"], case["nodes"], case["vocab"]
        target = torch.randn(b, n + 1, v, generator=g, device="cuda") * 3.5
        parents = np.stack([_parents(n, case["chain"], r) for _ in range(b)])
        up = torch.from_numpy(parents + 1).cuda()  # the target row that a node's token was drafted for
        wide = up[:, :, None]
        if case["chain"]:
            # a draft model near the target: tokens drawn from its own probabilities
            draft = target[:, :n] + 0.4 * torch.randn(b, n, v, generator=g, device="cuda")
            draft = torch.softmax(draft, -1)
            tokens = torch.multinomial(draft.view(b * n, v), 1, generator=g).view(b, n)
            s["draft_probs"] = draft.view(b * n, v)
        else:
            # the best candidates after every node, siblings in order
            rank = torch.from_numpy(np.stack([[int((row[:j] == row[j]).sum()) for j in range(n)] for row in parents])).cuda()
            best = torch.topk(target + 0.3 * torch.randn(b, n + 1, v, generator=g, device="cuda"), n, -1).indices
            tokens = best.gather(1, wide.expand(b, n, n)).gather(2, rank[:, :, None])[:, :, 0]
            s["draft_probs"] = None
        s["target_probs"] = torch.softmax(target, -1).view(b * (n + 1), v)
        s["tokens"] = tokens.to(torch.int32).reshape(-1).contiguous()
        s["parents"] = None if case["chain"] else torch.from_numpy(parents.astype(np.int32).reshape(-1)).cuda()
        s["node_offsets"] = torch.arange(0, b * n + 1, n, dtype=torch.int32, device="cuda")
        s["coins"] = torch.rand(b * (n + 1), generator=g, device="cuda")
        s["last_coins"] = torch.rand(b, generator=g, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        from mixture_experts_ffn_moe_gb300 import gbmoe
        return {"rope": _own_rope, "linear": _own_linear, "tree": _own_tree, "verify": _own_verify}[s["op"]](gbmoe, s)
    return {"rope": _plain_rope, "linear": _plain_linear, "tree": _plain_tree, "verify": _plain_verify}[s["op"]](s)


def _split(s):
    """q, k and v as views of the projections' output; without a cache, the part of the heads that turns."""
    hq, hk = s["q_heads"], s["k_heads"]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:]
    if not s["page"]:
        part = slice(s["offset"], s["offset"] + s["rot"])
        return q[..., part], k[..., part], v
    return q, k, v


def _own_rope(gbmoe, s):
    q, k, v = _split(s)
    if s["page"]:
        q_out = gbmoe.moe_rope_append(q, k, v, s["positions"], s["inv_freq"], s["slots"], s["k_cache"], s["v_cache"],
                                      scale=s["scale"], interleaved=s["interleaved"], inverse=s["inverse"],
                                      offset=s["offset"])
        return q_out, s["k_cache"], s["v_cache"]
    return gbmoe.moe_rope(q, k, s["positions"], s["inv_freq"], scale=s["scale"], interleaved=s["interleaved"],
                          inverse=s["inverse"])


def _plain_rope(s):
    q, k, v = _split(s)
    rot, lo = s["rot"], s["offset"] if s["page"] else 0
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    angle = -angle if s["inverse"] else angle
    cos, sin = (angle.cos() * s["scale"]).float()[:, None], (angle.sin() * s["scale"]).float()[:, None]

    def turn(x):
        part = x[..., lo:lo + rot].float()
        if s["interleaved"]:
            a, b = part[..., 0::2], part[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = part[..., :rot // 2], part[..., rot // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([x[..., :lo], y.to(x.dtype), x[..., lo + rot:]], -1)

    if not s["page"]:
        return turn(q), turn(k)
    put = s["slots"] >= 0
    at = s["slots"][put].long()
    s["k_cache"].view(-1, *k.shape[1:])[at] = turn(k)[put]
    s["v_cache"].view(-1, *v.shape[1:])[at] = v[put]
    return turn(q), s["k_cache"], s["v_cache"]


def _own_linear(gbmoe, s):
    return gbmoe.moe_linear_int4(s["x"], s["w"], s["w_scale"], gated=s["gated"])


def _plain_linear(s):
    w = s["w"]
    codes = torch.stack([w & 15, w >> 4], -1).flatten(1).float()
    codes = torch.where(codes > 7, codes - 16, codes)
    weight = (codes.view(w.shape[0], -1, s["group"]) * s["w_scale"][:, :, None]).view(codes.shape)
    y = s["x"].float() @ weight.T
    if s["gated"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(s["x"].dtype)


def _own_tree(gbmoe, s):
    return gbmoe.moe_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"],
                                    s["node_offsets"], s["tree_mask"])


def _plain_tree(s):
    q, offs, lens, page = s["q"], s["node_offsets"].long(), s["context_lens"].long(), s["page"]
    longest, widest = s["most"]
    hk, d, group = s["k_heads"], s["dim"], s["q_heads"] // s["k_heads"]
    at = torch.arange(longest, device=q.device)
    nodes = torch.arange(widest, device=q.device)
    batch = len(lens)
    have = nodes < (offs[1:] - offs[:-1])[:, None]
    row = torch.where(have, offs[:-1, None] + nodes, 0)
    # what every node sees: the committed slots, and the drafted ones whose bits its mask has
    node = at - lens[:, None]
    bit = (s["tree_mask"][row][:, :, None] >> node.clamp(0, 63)[:, None]) & 1
    drafted = (node >= 0) & (node < (offs[1:] - offs[:-1])[:, None])
    sees = (node < 0)[:, None] | (drafted[:, None] & (bit != 0))
    used = (node < 0) | drafted
    table = torch.where(used, s["block_table"].long()[:, at // page], 0)
    k = s["k_cache"][table, at % page].float().permute(0, 2, 1, 3)
    v = s["v_cache"][table, at % page].float().permute(0, 2, 1, 3) * used[:, None, :, None]
    wide = q[row].float().view(batch, widest, hk, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hk, widest * group, d)
    score = wide @ k.transpose(-1, -2) * d ** -0.5
    score = score.view(batch, hk, widest, group, longest).masked_fill_(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    y = p.view(batch, hk, widest * group, longest) @ v
    total = p.sum(-1).view(batch, hk, widest * group, 1)
    y = torch.where(total > 0, y / total, 0.0)
    y = y.view(batch, hk, widest, group, d).permute(0, 2, 1, 3, 4).reshape(batch, widest, hk * group, d)
    return y[have].to(q.dtype)


def _own_verify(gbmoe, s):
    return gbmoe.moe_verify_draft(s["target_probs"], s["tokens"], s["node_offsets"], s["coins"], s["last_coins"],
                                  s["nodes"], parents=s["parents"], draft_probs=s["draft_probs"])


def _plain_verify(s):
    b, n, v = s["batch"], s["nodes"], s["vocab"]
    target, tokens = s["target_probs"].view(b, n + 1, v), s["tokens"].view(b, n).long()
    coins = s["coins"].view(b, n + 1).double()
    j = torch.arange(n, device=tokens.device)
    up = (j - 1).expand(b, n) if s["parents"] is None else s["parents"].view(b, n).long()
    coin = coins.gather(1, up + 1)
    p = target[torch.arange(b, device=tokens.device)[:, None], up + 1, tokens].double()
    if s["draft_probs"] is not None:
        q = s["draft_probs"].view(b, n, v).gather(2, tokens[:, :, None])[:, :, 0].double()
        taken = coin * q < p
    else:
        # a parent's coin falls into the share of one child, or of none; a sibling's repeat has no share
        sibling = (up[:, :, None] == up[:, None, :]) & (j[None, :] < j[:, None])
        again = (sibling & (tokens[:, :, None] == tokens[:, None, :])).any(-1)
        p = torch.where(again, 0.0, p)
        before = (sibling * p[:, None, :]).sum(-1)
        taken = (coin >= before) & (coin < before + p) & ~again
    # accepted: taken, and so is every ancestor (doubling the reach, six steps cover 64 nodes)
    ok, far = taken, up
    ok, far = _lift(ok, far)
    ok, far = _lift(ok, far)
    ok, far = _lift(ok, far)
    ok, far = _lift(ok, far)
    ok, far = _lift(ok, far)
    ok, far = _lift(ok, far)
    count = ok.sum(-1)
    path = torch.sort(torch.where(ok, j, n), -1).values
    stop = torch.where(count > 0, path.gather(1, (count - 1).clamp(min=0)[:, None])[:, 0], -1)
    rows = torch.arange(b, device=tokens.device)
    w = target[rows, stop + 1].double()
    if s["draft_probs"] is not None:
        # a refused token leaves what the target has more than the draft
        q = s["draft_probs"].view(b, n, v)[rows, (stop + 1).clamp(max=n - 1)].double()
        w = torch.where((stop + 1 < n)[:, None], (w - q).clamp(min=0.0), w)
    else:
        # refused children leave the rest
        child = up == stop[:, None]
        gone = torch.zeros(b, v, dtype=torch.bool, device=w.device)
        gone.view(-1).index_fill_(0, (rows[:, None] * v + tokens)[child], True)
        w = torch.where(gone, 0.0, w)
    whole = w.cumsum(-1)
    level = s["last_coins"].double()[:, None] * whole[:, -1:]
    last = (whole > level).to(torch.int8).argmax(-1)
    path = torch.where(path < n, path, -1)
    out = torch.where(path >= 0, tokens.gather(1, path.clamp(min=0)), -1)
    out = torch.cat([out, torch.full_like(out[:, :1], -1)], 1).scatter(1, count[:, None], last[:, None])
    return out.int(), path.int(), count.int()


def _lift(ok, far):
    up = far.clamp(min=0)
    return ok & (ok.gather(1, up) | (far < 0)), torch.where(far < 0, far, far.gather(1, up))


# ------------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "linear": _exact_linear, "tree": _exact_tree, "verify": _exact_verify}[case["op"]](s)


def _exact_rope(s):
    """Pairs as complex numbers, times scale * exp(i * angle)."""
    f, scale = _frequencies(s)
    angle = s["positions"].cpu().numpy().astype(np.float64)[:, None] * f
    z = torch.from_numpy(scale * np.exp((-1j if s["inverse"] else 1j) * angle)).cuda()[:, None, :]
    rot, half = s["rot"], s["rot"] // 2
    lo = s["offset"]
    a = np.arange(half)
    first, second = (lo + 2 * a, lo + 2 * a + 1) if s["interleaved"] else (lo + a, lo + half + a)
    hq, hk = s["q_heads"], s["k_heads"]
    x = s["qkv"][:, :hq + hk].double()
    turned = x.clone()
    pair = torch.complex(x[..., first], x[..., second]) * z
    turned[..., first], turned[..., second] = pair.real, pair.imag
    if not s["page"]:
        turned = turned[..., lo:lo + rot]
        return turned[:, :hq], turned[:, hq:]
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            k_cache[slot // s["page"], slot % s["page"]] = turned[t, hq:]
            v_cache[slot // s["page"], slot % s["page"]] = s["qkv"][t, hq + hk:].double()
    return turned[:, :hq], k_cache, v_cache


def _exact_linear(s):
    m, n = s["rows"], s["w"].shape[0]
    x = s["x"].double()
    low, high = x[:, 0::2], x[:, 1::2]
    y = torch.empty(m, n, dtype=torch.float64, device=x.device)
    for at in range(0, n, 4096):
        w = s["w"][at:at + 4096].to(torch.int16)
        scale = s["w_scale"][at:at + 4096].double().repeat_interleave(s["group"] // 2, 1)
        y[:, at:at + 4096] = (low @ ((((w & 15) ^ 8) - 8).double() * scale).T
                              + high @ ((((w >> 4) ^ 8) - 8).double() * scale).T)
    if s["gated"]:
        y = torch.nn.functional.silu(y[:, :s["outer"]]) * y[:, s["outer"]:]
    return y


def _exact_tree(s):
    page, d, group = s["page"], s["dim"], s["q_heads"] // s["k_heads"]
    offs, lens = s["node_offsets"].tolist(), s["context_lens"].tolist()
    masks = s["tree_mask"].cpu().numpy().view(np.uint64)
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        lo, hi = offs[b], offs[b + 1]
        whole = length + hi - lo
        slots = torch.cat([page * p + torch.arange(page, device="cuda") for p in s["block_table"][b, :-(-whole // page)].long()])[:whole]
        hide = torch.zeros(hi - lo, whole, device="cuda", dtype=torch.bool)
        hide[:, length:] = torch.from_numpy(((masks[lo:hi, None] >> np.arange(hi - lo, dtype=np.uint64)) & np.uint64(1)) == 0).cuda()
        for h in range(s["k_heads"]):
            k = s["k_cache"][slots // page, slots % page, h].double()
            v = s["v_cache"][slots // page, slots % page, h].double()
            for x in range(h * group, (h + 1) * group):
                score = (s["q"][lo:hi, x].double() @ k.T / math.sqrt(d)).masked_fill(hide, -math.inf)
                y[lo:hi, x] = torch.nan_to_num(torch.softmax(score, -1), nan=0.0) @ v
    return y


def _exact_verify(s):
    """Walks every tree from its root."""
    n = s["nodes"]
    tokens = s["tokens"].tolist()
    coins, last = s["coins"].double().cpu().numpy(), s["last_coins"].double().cpu().numpy()
    out, path, count = (np.full((s["batch"], n + 1), -1), np.full((s["batch"], n), -1), np.zeros(s["batch"], dtype=np.int64))
    for b in range(s["batch"]):
        up = list(range(-1, n - 1)) if s["parents"] is None else s["parents"][b * n:(b + 1) * n].tolist()
        token = tokens[b * n:(b + 1) * n]
        node = -1
        while True:
            row = s["target_probs"][b * (n + 1) + node + 1].double().cpu().numpy()
            coin = coins[b * (n + 1) + node + 1]
            children = [j for j in range(n) if up[j] == node]
            found = None
            if s["draft_probs"] is None:
                share = 0.0
                for i, j in enumerate(children):
                    if token[j] not in [token[c] for c in children[:i]]:
                        if share <= coin < share + row[token[j]]:
                            found = j
                            break
                        share += row[token[j]]
                if found is None:
                    row[[token[j] for j in children]] = 0.0
            elif children:
                q = s["draft_probs"][b * n + children[0]].double().cpu().numpy()
                if coin * q[token[children[0]]] < row[token[children[0]]]:
                    found = children[0]
                else:
                    row = np.maximum(row - q, 0.0)
            if found is None:
                break
            out[b, count[b]], path[b, count[b]] = token[found], found
            count[b] += 1
            node = found
        whole = np.cumsum(row)
        out[b, count[b]] = int(np.argmax(whole > last[b] * whole[-1]))
    return torch.from_numpy(out).int(), torch.from_numpy(path).int(), torch.from_numpy(count).int()
