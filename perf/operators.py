"""The draft-tree operators over the paged KV cache: what is measured of them, and their plain forms.

A step of speculative decoding gives every sequence a small tree of drafted
tokens behind its ctx cached ones (a node's parent is an earlier node of the
same sequence, -1 stands for the last cached token; node i takes cache slot
ctx + i and position ctx + depth(i)).  Three operators carry it:

* append: per-head RMSNorm (optional) and rotary positions of the queries and
  keys of all nodes, and the keys and values written into the paged cache;
* attend: every node attends to its sequence's cached tokens, its ancestors
  and itself, over the pages;
* commit: the walk down the tree along the tokens the model chose, and the
  accepted nodes' keys and values moved, in every layer, to where a plain
  sequence would have them.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
EPS = 1e-6
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases ---------------------------------------------------------------------------------------------


def listed():
    big = {"heads": 16, "kv_heads": 8, "head_dim": 128, "cache": "f16"}
    mid = {"heads": 8, "kv_heads": 4, "head_dim": 64, "cache": "f32"}
    rope = {"layout": "half", "rot": 128, "scaling": "none", "norm": True, "in": "f32", "q_out": "f32"}
    return [
        # one new token of one sequence, straight from the QKV product: nothing but latency
        {"name": "append 1x1", "op": "append", **big, **rope, "seqs": 1, "tokens": 1, "ctx_lo": 500, "ctx_hi": 500, "tree": "chain"},
        # the drafted trees of a serving batch, bf16 projections, half of each head rotated, scaled for a long context
        {"name": "append 32x17 bf16", "op": "append", **big, "layout": "interleaved", "rot": 64, "scaling": "yarn", "norm": False, "in": "bf16", "q_out": "bf16",
         "seqs": 32, "tokens": 17, "ctx_lo": 100, "ctx_hi": 900, "tree": "random"},
        # the widest step: 32 sequences of 256 nodes each, as a chunk of prompt takes it
        {"name": "append 32x256", "op": "append", **big, **rope, "seqs": 32, "tokens": 256, "ctx_lo": 0, "ctx_hi": 200, "tree": "chain"},
        # the full-precision cache of the parity mode, odd sizes
        {"name": "append 5x33 f32", "op": "append", **mid, **rope, "rot": 48, "scaling": "bands", "seqs": 5, "tokens": 33, "ctx_lo": 7, "ctx_hi": 333, "tree": "random"},
        # a short draft of one sequence: the smallest verification
        {"name": "attend 1x5 ctx 500", "op": "attend", **big, "in": "f32", "out": "bf16", "seqs": 1, "tokens": 5, "ctx_lo": 500, "ctx_hi": 500, "tree": "chain"},
        # one sequence at the longest context that the decoder takes, a wide tree
        {"name": "attend 1x64 ctx 40000", "op": "attend", **big, "in": "f32", "out": "bf16", "seqs": 1, "tokens": 64, "ctx_lo": 40000, "ctx_hi": 40000, "tree": "random"},
        # the serving batch, 8 drafted tokens each: bound by the cache's bytes
        {"name": "attend 32x8 ctx 1024-2048", "op": "attend", **big, "in": "f32", "out": "bf16", "seqs": 32, "tokens": 8, "ctx_lo": 1024, "ctx_hi": 2048, "tree": "random"},
        # the same batch with trees of 64: bytes and products near balance
        {"name": "attend 32x64 ctx 1024-2048", "op": "attend", **big, "in": "bf16", "out": "bf16", "seqs": 32, "tokens": 64, "ctx_lo": 1024, "ctx_hi": 2048, "tree": "random"},
        # the widest trees over long contexts: bound by the products
        {"name": "attend 8x256 ctx 8000", "op": "attend", **big, "in": "f32", "out": "bf16", "seqs": 8, "tokens": 256, "ctx_lo": 7800, "ctx_hi": 8200, "tree": "random"},
        # the full-precision cache of the parity mode, ragged
        {"name": "attend 5x33 ctx 777 f32", "op": "attend", **mid, "in": "f32", "out": "f32", "seqs": 5, "tokens": 33, "ctx_lo": 111, "ctx_hi": 777, "tree": "random"},
        # one sequence's accepted path, 28 layers
        {"name": "commit 1x16 28 layers", "op": "commit", **big, "layers": 28, "seqs": 1, "tokens": 16, "ctx_lo": 300, "ctx_hi": 300, "tree": "random", "accept": 5},
        # a serving batch's accepted paths
        {"name": "commit 32x64 28 layers", "op": "commit", **big, "layers": 28, "seqs": 32, "tokens": 64, "ctx_lo": 0, "ctx_hi": 100, "tree": "random", "accept": 9},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 0.7)), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attend", "attend", "commit"])
        heads, kv = rng.choice([(4, 2), (8, 4), (16, 8), (8, 8), (16, 4), (32, 8), (12, 3), (5, 5)])
        c = {"op": op, "heads": heads, "kv_heads": kv, "head_dim": rng.choice([32, 64, 128, 128]), "cache": rng.choice(["f16", "f16", "f16", "f32"]),
             "seqs": _log_int(rng, 1, 33), "tokens": _log_int(rng, 1, 256), "tree": rng.choice(["chain", "random", "random"])}
        c["ctx_lo"] = _log_int(rng, 1, 40000 if op == "attend" else 1000) - 1
        c["ctx_hi"] = min(40000, c["ctx_lo"] + _log_int(rng, 1, 1000) - 1)
        width, nodes, held = kv * c["head_dim"], c["seqs"] * c["tokens"], c["seqs"] * (c["ctx_hi"] + c["tokens"] + BLOCK)
        if op == "attend":
            c["in"] = rng.choice(["f32", "bf16", "f16"])
            c["out"] = "f32" if c["cache"] == "f32" else rng.choice(["bf16", "bf16", "f16"])
            # no more cache, scores or products than the largest listed attention; products in full precision run at a fraction of the rate
            if held * width > 72e6 or held * heads * c["tokens"] > 2.8e8 or held * heads * c["head_dim"] * c["tokens"] > (3.4e10 if c["cache"] == "f16" else 2e9):
                continue
        elif op == "append":
            c["layout"] = rng.choice(["half", "interleaved"])
            c["rot"] = rng.randrange(8, c["head_dim"] + 1, 8)
            c["scaling"] = rng.choice(["none", "linear", "yarn", "bands"])
            c["norm"] = rng.random() < 0.5
            c["in"], c["q_out"] = rng.choice(["f32", "bf16", "f16"]), rng.choice(["f32", "f32", "bf16"])
            if nodes * (heads + 2 * kv) * c["head_dim"] > 33e6 or held * width > 30e6:
                continue
        else:
            c["layers"] = rng.choice([2, 8, 28])
            c["accept"] = rng.randint(1, min(c["tokens"], 12))
            if held * width * c["layers"] > 2.4e8 or nodes * width > 2.4e6:
                continue
        return c


# ---- what a program holds before the call -------------------------------------------------------------------


def _layers(case):
    return case.get("layers", 2)


def _sizes(case):
    """Contexts and node counts of the sequences; a batch is ragged, the first sequence has the full count."""
    s, t = case["seqs"], case["tokens"]
    ctx = [case["ctx_lo"] + (i * (case["ctx_hi"] - case["ctx_lo"])) // max(s - 1, 1) for i in range(s)]
    return ctx, [max(1, t - (i * 5) % (t // 4 + 1)) for i in range(s)]


def _parents(case, count, rng):
    """A chain, or a tree whose nodes mostly hang near its root (node 0 is the sampled, certain token)."""
    if case["tree"] == "chain":
        return [i - 1 for i in range(count)]
    return [-1] + [max(0, min(i - 1, int(i * rng.random() ** 1.5))) for i in range(1, count)]


def _frequencies(case):
    """Rotary frequencies per pair and the factor on cos and sin, in 64 bits."""
    rot, base, orig, factor = case["rot"], 1e6, 4096, 4.0
    f = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "yarn":
        low, high = (rot * math.log(orig / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = [min(max((j - low) / max(high - low, 0.001), 0.0), 1.0) for j in range(rot // 2)]
        return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "bands":
        smooth = [min(max((orig * x / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0), 1.0) for x in f]
        return [x * s + x / factor * (1 - s) for x, s in zip(f, smooth)], 1.0
    return f, 1.0


def prepare(case, seed):
    rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    H, Hkv, D, L, S = case["heads"], case["kv_heads"], case["head_dim"], _layers(case), case["seqs"]
    ctx, counts = _sizes(case)
    parents = [_parents(case, n, rng) for n in counts]
    N, T, longest = sum(counts), max(counts), max(c + n for c, n in zip(ctx, counts))
    need = [(c + n + BLOCK - 1) // BLOCK for c, n in zip(ctx, counts)]
    blocks = sum(need) + 3
    order = list(range(blocks))
    rng.shuffle(order)  # pages lie anywhere in the pool
    tables, at = [], 0
    for n in need:
        tables.append(order[at:at + n])
        at += n
    slab = torch.randn((L, blocks, 2, Hkv, BLOCK, D), generator=g, device="cuda", dtype=torch.float32 if L * blocks * Hkv * D < 1 << 22 else torch.float16)
    slab = slab.to(TYPES[case["cache"]])

    # what the plain form goes by: page and slot of each key, which node sees which key, the padded nodes
    table = np.zeros((S, max(need)), dtype=np.int64)
    nodes, starts, depth = np.full((S, T), N, dtype=np.int64), np.cumsum([0] + counts), np.zeros(N, dtype=np.int64)
    up = np.full((S, T), -2, dtype=np.int64)
    sees = np.zeros((S, T, T), dtype=bool)
    for s in range(S):
        table[s, :need[s]] = tables[s]
        nodes[s, :counts[s]] = starts[s] + np.arange(counts[s])
        up[s, :counts[s]] = parents[s]
        for i, p in enumerate(parents[s]):
            if p >= 0:
                sees[s, i] = sees[s, p]
                depth[starts[s] + i] = depth[starts[s] + p] + 1
            sees[s, i, i] = True
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    tab, ctx_t = dev(table), dev(np.array(ctx, dtype=np.int64))
    seq = dev(np.repeat(np.arange(S), counts))
    index = dev(np.concatenate([np.arange(n) for n in counts]))
    slot = ctx_t[seq] + index
    st = {"op": case["op"], "H": H, "Hkv": Hkv, "D": D, "layer": L - 1, "slab": slab, "nodes": dev(nodes), "seq": seq, "index": index, "N": N}
    st |= {"block": tab[seq, slot // BLOCK], "slot": slot % BLOCK}

    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "append":
        # one buffer of raw q|k|v rows, as the QKV product leaves it
        raw = rand(N, (H + 2 * Hkv) * D).to(TYPES[case["in"]])
        st["q"], st["k"], st["v"] = (x.view(N, -1, D) for x in raw.split([H * D, Hkv * D, Hkv * D], dim=1))
        st["q_norm"], st["k_norm"] = (1 + 0.1 * rand(D), 1 + 0.1 * rand(D)) if case["norm"] else (None, None)
        freq, mult = _frequencies(case)
        angle = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(freq, device="cuda", dtype=torch.float64)
        st["cos"], st["sin"] = (angle.cos() * mult).float(), (angle.sin() * mult).float()
        st["position"], st["half"], st["rot"] = ctx_t[seq] + dev(depth), case["layout"] == "half", case["rot"]
        st["q_type"] = TYPES[case["q_out"]]
    elif case["op"] == "attend":
        st["q"] = rand(N, H, D).to(TYPES[case["in"]])
        st["out_type"] = TYPES[case["out"]]
        key = torch.arange(longest, device="cuda")
        st["key_block"], st["key_slot"] = tab[:, key // BLOCK], key % BLOCK
        rel = key[None] - ctx_t[:, None]  # [S, keys]: negative for cached tokens, else the node's number
        seen = torch.gather(dev(sees), 2, rel.clamp(0, T - 1)[:, None].expand(S, T, longest)) & (rel < T)[:, None]
        st["sees"] = torch.where(rel[:, None] < 0, True, seen)
    else:
        vocab = 151936
        draft = torch.randint(vocab, (N,), generator=g, device="cuda", dtype=torch.int32)
        target = torch.randint(vocab, (N,), generator=g, device="cuda", dtype=torch.int32)
        for s in range(S):  # the model agrees with the draft down to `accept` nodes, or to a leaf before
            children = [[] for _ in range(counts[s])]
            for i, p in enumerate(parents[s]):
                if p >= 0:
                    children[p].append(i)
            at, steps, b = 0, 1, int(starts[s])
            while children[at] and steps < case["accept"]:
                to = rng.choice(children[at])
                target[b + at] = draft[b + to]
                at, steps = to, steps + 1
        st["draft"], st["target"] = draft, target
        st["up"], st["sees"], st["ctx"], st["tab"], st["S"] = dev(up), dev(sees), ctx_t, tab, S
    if own:  # the program's cache pool, its rotary table and the plan of this step's trees, kept over the layers
        from decoder_qwen3_step_gb300 import dec
        from decoder_qwen3_step_gb300.trees import DraftTrees, KvPool, RopeTable

        shape = {"vocab": 512, "d_model": 64, "n_layers": L, "n_heads": H, "n_kv_heads": Hkv, "head_dim": D, "ff_hidden": 64}
        pool = KvPool(shape, dec.DEC_FP32 if case["cache"] == "f32" else dec.DEC_BF16_F16KV, blocks, max_positions=40960, slabs=slab)
        pool.alloc(blocks)
        st["trees"] = DraftTrees(pool, max_seqs=S, max_tokens=N, max_blocks=max(need))
        st["trees"].set(ctx, parents, tables)
        if case["op"] == "append":
            kinds = {"none": dec.DEC_ROPE_PLAIN, "linear": dec.DEC_ROPE_LINEAR, "yarn": dec.DEC_ROPE_YARN, "bands": dec.DEC_ROPE_BANDS}
            more = {"yarn": {"low": 1.0, "high": 32.0, "attn_factor": 0.1 * math.log(4.0) + 1.0}, "bands": {"low": 1.0, "high": 4.0}}.get(case["scaling"], {})
            st["rope"] = RopeTable(case["rot"], longest, base=1e6, layout=dec.DEC_ROPE_HALF if st["half"] else dec.DEC_ROPE_INTERLEAVED, scaling=kinds[case["scaling"]],
                                   factor=4.0, orig_positions=4096, **more)
    return st


# ---- one pass -------------------------------------------------------------------------------------------------


def _rotated(x, gain, st):
    """Per-head RMSNorm where a gain is given, then the rotation of the first `rot` channels."""
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    rot = st["rot"]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if st["half"] else (x[..., 0:rot:2], x[..., 1:rot:2])
    c, s = st["cos"][st["position"]][:, None], st["sin"][st["position"]][:, None]
    a, b = a * c - b * s, b * c + a * s
    turned = torch.cat([a, b], -1) if st["half"] else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _append(st):
    slab, layer = st["slab"], st["layer"]
    q = _rotated(st["q"], st["q_norm"], st).to(st["q_type"])
    slab[layer, st["block"], 0, :, st["slot"]] = _rotated(st["k"], st["k_norm"], st).to(slab.dtype)
    slab[layer, st["block"], 1, :, st["slot"]] = st["v"].to(slab.dtype)
    return {"q": q, "cache": slab}


def _attend(st):
    H, Hkv, D = st["H"], st["Hkv"], st["D"]
    kv = st["slab"][st["layer"]][st["key_block"], :, :, st["key_slot"]].float()  # [S, keys, 2, Hkv, D]
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    q = torch.cat([st["q"].float(), st["q"].new_zeros(1, H, D).float()])[st["nodes"]]  # [S, T, H, D], zeros where a sequence has no such node
    S, T = q.shape[:2]
    q = q.view(S, T, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, T * (H // Hkv), D)
    s = (q @ k.transpose(2, 3) / math.sqrt(D)).view(S, Hkv, T, H // Hkv, -1)
    s = s.masked_fill(~st["sees"][:, None, :, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    o = (p.view(S, Hkv, T * (H // Hkv), -1) @ v).view(S, Hkv, T, H // Hkv, D) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.permute(0, 2, 1, 3, 4).reshape(S, T, H * D)[st["seq"], st["index"]].to(st["out_type"])


def _commit(st):
    nodes, up, ctx, tab, slab = st["nodes"], st["up"], st["ctx"], st["tab"], st["slab"]
    S, T = nodes.shape
    pad = lambda x: torch.cat([x, x.new_full((1,), -1)])[nodes]  # noqa: E731
    draft, target = pad(st["draft"]), pad(st["target"])
    right = (up >= 0) & (draft == torch.gather(target, 1, up.clamp(min=0))) | (up == -1)  # as the parent's choice; the root is certain
    earlier = (up[:, :, None] == up[:, None, :]) & torch.ones(T, T, dtype=torch.bool, device=up.device).tril(-1) & right[:, None, :]
    right = right & ~earlier.any(-1)
    taken = ~(st["sees"] & ~right[:, None, :]).any(-1) & (up >= -1)  # the whole way from the root
    n = taken.sum(-1)
    at = torch.arange(T, device=up.device)
    path = torch.where(taken, at, T).sort(-1).values
    good = at < n[:, None]
    frm = torch.where(good, path, at)  # a node that is not on the path stays as it is
    have = nodes < st["N"]
    src, dst, seq = (ctx[:, None] + frm)[have], (ctx[:, None] + at)[have], st["seq"]
    slab[:, tab[seq, dst // BLOCK], :, :, dst % BLOCK] = slab[:, tab[seq, src // BLOCK], :, :, src % BLOCK]
    last = torch.gather(path, 1, (n - 1)[:, None])
    return {"accepted": n.int(), "path": torch.where(good, path, -1)[have].int(), "next": torch.gather(target, 1, last)[:, 0], "cache": slab}


def run(st):
    if own:
        trees = st["trees"]
        if st["op"] == "append":
            q = trees.append(st["layer"], st["q"], st["k"], st["v"], rope=st["rope"], q_norm=st["q_norm"], k_norm=st["k_norm"], q_type=st["q_type"])
            return {"q": q, "cache": st["slab"]}
        if st["op"] == "attend":
            return trees.attend(st["layer"], st["q"], out_type=st["out_type"])
        accepted, path, after = trees.commit(st["draft"], st["target"])
        return {"accepted": accepted, "path": path, "next": after, "cache": st["slab"]}
    return {"append": _append, "attend": _attend, "commit": _commit}[st["op"]](st)


# ---- what a pass cannot do without ----------------------------------------------------------------------------


def work(case):
    ctx, counts = _sizes(case)
    H, Hkv, D, N = case["heads"], case["kv_heads"], case["head_dim"], sum(counts)
    size = {"f32": 4, "f16": 2, "bf16": 2}
    cache = size[case["cache"]]
    if case["op"] == "append":
        width = size[case["in"]]
        moved = N * D * (H * (width + size[case["q_out"]]) + 2 * Hkv * (width + cache)) + N * case["rot"] * 4
        return {"bytes": moved, "flops": N * (H + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    if case["op"] == "attend":
        keys = sum(c + n for c, n in zip(ctx, counts))
        return {"bytes": 2 * keys * Hkv * D * cache + N * H * D * (size[case["in"]] + size[case["out"]]), "flops": sum(4 * D * H * n * (c + n / 2) for c, n in zip(ctx, counts))}
    rows = sum(max(min(case["accept"], n) - 1, 0) for n in counts)
    rows = 0 if case["tree"] == "chain" else rows  # a chain's accepted nodes are in place
    return {"bytes": 4 * rows * _layers(case) * Hkv * D * cache + 16 * N, "flops": 4 * N}


# ---- the definition, in 64 bits --------------------------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    ctx, counts = _sizes(case)
    H, Hkv, D, layer = st["H"], st["Hkv"], st["D"], st["layer"]
    if case["op"] == "append":
        freq, mult = _frequencies(case)
        angle = st["position"].double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full_like(angle, mult), angle)  # each pair as a complex number

        def formed(x, gain):
            x = x.double()
            if gain is not None:
                x = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * gain.double()
            y, rot = x.clone(), case["rot"]
            first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if st["half"] else (slice(0, rot, 2), slice(1, rot, 2))
            z = torch.complex(x[..., first], x[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        cache = st["slab"].double()
        for is_v, rows in ((0, formed(st["k"], st["k_norm"])), (1, st["v"].double())):
            flat = cache[layer, :, is_v]
            flat[st["block"], :, st["slot"]] = rows
        return {"q": formed(st["q"], st["q_norm"]), "cache": cache}
    if case["op"] == "attend":
        if sum(4 * D * H * n * (c + n) for c, n in zip(ctx, counts)) > 4e11:
            return None
        out = torch.empty((st["N"], H, D), dtype=torch.float64, device="cuda")
        b = 0
        for s, (c, n) in enumerate(zip(ctx, counts)):
            rows = st["slab"][layer][st["key_block"][s, :c + n], :, :, st["key_slot"][:c + n]].double()  # [keys, 2, Hkv, D]
            for h in range(H):
                kv = rows[:, :, h * Hkv // H]
                score = st["q"][b:b + n, h].double() @ kv[:, 0].T * D ** -0.5
                weight = torch.softmax(torch.where(st["sees"][s, :n, :c + n], score, -math.inf), dim=-1)
                out[b:b + n, h] = weight @ kv[:, 1]
            b += n
        return out.flatten(1)
    # commit moves what is there: the walk and the move, node by node
    cache, b = st["slab"].double(), 0
    draft, target, up, tab = (st[k].tolist() for k in ("draft", "target", "up", "tab"))
    accepted, path, after = [], [], []
    for s, n in enumerate(counts):
        at, way = 0, [0]
        while True:
            to = [i for i in range(n) if up[s][i] == at and draft[b + i] == target[b + at]]
            if not to:
                break
            at = to[0]
            way.append(at)
        places = [(tab[s][(ctx[s] + i) // BLOCK], (ctx[s] + i) % BLOCK) for i in range(n)]
        for i, w in enumerate(way):
            if w != i:
                cache[:, places[i][0], :, :, places[i][1]] = cache[:, places[w][0], :, :, places[w][1]]
        accepted.append(len(way))
        path += way + [-1] * (n - len(way))
        after.append(target[b + at])
        b += n
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"accepted": whole(accepted), "path": whole(path), "next": whole(after), "cache": cache}
