"""The operators over a paged KV cache held in 8 bits: what is measured of them, and their plain forms.

A page (the K or the V of 16 slots of one KV head) holds 8-bit codes and one
scale 2^e; a value is code * 2^e.  Codes are whole numbers -127 .. 127 or e4m3
numbers up to 448 (Q below).  Four operators carry it:

* append: per-head RMSNorm (optional) and rotary positions of the queries and
  keys of all nodes, and the keys and values quantised into the cache.  e is
  the smallest of -40 .. 40 with (largest magnitude) <= Q 2^e over the rows that
  the call writes to the page, and, where the page holds earlier tokens, not
  below the page's e so far; if it rises, the earlier tokens' codes are rounded
  again to the new scale.  Codes round to nearest even;
* attend: every node of a draft tree attends to its sequence's cached tokens,
  its ancestors and itself, over the pages;
* commit: the walk down the tree along the tokens the model chose, and the
  accepted nodes' keys and values moved, in every layer, to where a plain
  sequence would have them, quantised to the page they move to;
* read: keys and values of sequences read back from the pages.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
EPS = 1e-6
E_MIN, E_MAX = -40, 40
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---- the cases ---------------------------------------------------------------------------------------------


def listed():
    big = {"heads": 16, "kv_heads": 8, "head_dim": 128}
    rope = {"layout": "half", "rot": 128, "scaling": "none", "norm": True, "in": "f32", "q_out": "f32"}
    return [
        # one new token of one sequence in the middle of a page, straight from the QKV product: nothing but latency
        {"name": "append 1x1 i8", "op": "append", **big, **rope, "codes": "i8", "seqs": 1, "tokens": 1, "ctx_lo": 501, "ctx_hi": 501, "tree": "chain"},
        # the drafted trees of a serving batch, bf16 projections, half of each head rotated, scaled for a long context
        {"name": "append 32x17 e4m3 bf16", "op": "append", **big, "layout": "interleaved", "rot": 64, "scaling": "yarn", "norm": False, "in": "bf16", "q_out": "bf16",
         "codes": "e4m3", "seqs": 32, "tokens": 17, "ctx_lo": 100, "ctx_hi": 900, "tree": "random"},
        # the widest step: 32 sequences of 256 nodes each, as a chunk of prompt takes it
        {"name": "append 32x256 i8", "op": "append", **big, **rope, "codes": "i8", "seqs": 32, "tokens": 256, "ctx_lo": 0, "ctx_hi": 200, "tree": "chain"},
        # a short draft of one sequence: the smallest verification
        {"name": "attend 1x5 ctx 500 i8", "op": "attend", **big, "codes": "i8", "in": "f32", "out": "bf16", "seqs": 1, "tokens": 5, "ctx_lo": 500, "ctx_hi": 500, "tree": "chain"},
        # the decode step of the serving batch: bound by the cache's bytes
        {"name": "attend 32x1 ctx 1024-2048 i8", "op": "attend", **big, "codes": "i8", "in": "f32", "out": "bf16", "seqs": 32, "tokens": 1, "ctx_lo": 1024, "ctx_hi": 2048, "tree": "chain"},
        # one sequence at the longest context that the decoder takes, a wide tree
        {"name": "attend 1x64 ctx 40000 e4m3", "op": "attend", **big, "codes": "e4m3", "in": "f32", "out": "bf16", "seqs": 1, "tokens": 64, "ctx_lo": 40000, "ctx_hi": 40000, "tree": "random"},
        # the serving batch with trees of 64: bytes and products near balance
        {"name": "attend 32x64 ctx 1024-2048 i8", "op": "attend", **big, "codes": "i8", "in": "bf16", "out": "bf16", "seqs": 32, "tokens": 64, "ctx_lo": 1024, "ctx_hi": 2048, "tree": "random"},
        # the widest trees over long contexts: bound by the products
        {"name": "attend 8x256 ctx 8000 e4m3", "op": "attend", **big, "codes": "e4m3", "in": "f32", "out": "bf16", "seqs": 8, "tokens": 256, "ctx_lo": 7800, "ctx_hi": 8200, "tree": "random"},
        # a short sequence of a small model, read back to be looked at in full precision
        {"name": "read 1x100 f32 e4m3", "op": "read", "heads": 8, "kv_heads": 4, "head_dim": 64, "codes": "e4m3", "out": "f32", "layers": 1, "seqs": 1, "tokens": 1, "ctx_lo": 100, "ctx_hi": 100, "tree": "chain"},
        # the serving batch's sequences in all layers, for a program that moves them to an f16 cache
        {"name": "read 32x1024-2048 28 layers i8", "op": "read", **big, "codes": "i8", "out": "f16", "layers": 28, "seqs": 32, "tokens": 1, "ctx_lo": 1024, "ctx_hi": 2048, "tree": "chain"},
        # one sequence's accepted path, 28 layers, and the pages that it changed
        {"name": "commit 1x16 28 layers e4m3", "op": "commit", **big, "codes": "e4m3", "out": "bf16", "layers": 28, "seqs": 1, "tokens": 16, "ctx_lo": 300, "ctx_hi": 300, "tree": "random", "accept": 5},
        # a serving batch's accepted paths, and the pages that they changed
        {"name": "commit 32x64 28 layers i8", "op": "commit", **big, "codes": "i8", "out": "bf16", "layers": 28, "seqs": 32, "tokens": 64, "ctx_lo": 0, "ctx_hi": 100, "tree": "random", "accept": 9},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 0.7)), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attend", "attend", "attend", "commit", "read"])
        heads, kv = rng.choice([(4, 2), (8, 4), (16, 8), (8, 8), (16, 4), (32, 8), (12, 3), (5, 5)])
        c = {"op": op, "heads": heads, "kv_heads": kv, "head_dim": rng.choice([32, 64, 128, 128]), "codes": rng.choice(["i8", "e4m3"]),
             "seqs": _log_int(rng, 1, 33), "tokens": _log_int(rng, 1, 256), "tree": rng.choice(["chain", "random", "random"])}
        c["ctx_lo"] = _log_int(rng, 1, 40000 if op in ("attend", "read") else 1000) - 1
        c["ctx_hi"] = min(40000, c["ctx_lo"] + _log_int(rng, 1, 1000) - 1)
        width, nodes, held = kv * c["head_dim"], c["seqs"] * c["tokens"], c["seqs"] * (c["ctx_hi"] + c["tokens"] + BLOCK)
        if op == "attend":
            c["in"] = rng.choice(["f32", "bf16", "f16"])
            c["out"] = rng.choice(["bf16", "bf16", "f16"])
            # no more cache, scores or products than the largest listed attention
            if held * width > 72e6 or held * heads * c["tokens"] > 2.8e8 or held * heads * c["head_dim"] * c["tokens"] > 3.4e10:
                continue
        elif op == "append":
            c["layout"] = rng.choice(["half", "interleaved"])
            c["rot"] = rng.randrange(8, c["head_dim"] + 1, 8)
            c["scaling"] = rng.choice(["none", "linear", "yarn", "bands"])
            c["norm"] = rng.random() < 0.5
            c["in"], c["q_out"] = rng.choice(["f32", "bf16", "f16"]), rng.choice(["f32", "f32", "bf16"])
            if nodes * (heads + 2 * kv) * c["head_dim"] > 33e6 or held * width > 30e6:
                continue
        elif op == "read":
            c["layers"] = rng.choice([1, 2, 8, 28])
            c["out"] = rng.choice(["bf16", "f16", "f32"])
            if held * width * c["layers"] * (1 + SIZE[c["out"]]) > 5.6e9:
                continue
        else:
            c["layers"] = rng.choice([2, 8, 28])
            c["out"] = "bf16"
            c["accept"] = rng.randint(1, min(c["tokens"], 12))
            if held * width * c["layers"] > 1.4e8 or nodes * width > 2.4e6:
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


def _cache(case, blocks, g):
    """A buffer of codes [layers, blocks, 2, KV heads, 16, D] and, behind them, scales [layers, blocks, KV heads, 2] in f32."""
    L, H, D = _layers(case), case["kv_heads"], case["head_dim"]
    n = L * blocks * 2 * H * BLOCK * D
    at = (n + 255) // 256 * 256
    buf = torch.zeros(at + L * blocks * H * 2 * 4, dtype=torch.uint8, device="cuda")
    codes, scales = buf[:n].view(L, blocks, 2, H, BLOCK, D), buf[at:].view(torch.float32).view(L, blocks, H, 2)
    # a few channels of the keys stand out, as they do in trained models; pages differ in size
    gain = torch.ones((2, H, 1, D), device="cuda")
    gain[0, :, :, :: max(D // 4, 1)] = 5.0
    for layer in range(L):
        x = torch.randn((blocks, 2, H, BLOCK, D), generator=g, device="cuda") * gain
        x *= _two(torch.randint(-1, 2, (blocks, 2, H, 1, 1), generator=g, device="cuda"))
        e = _exponent(x.abs().amax((-2, -1)), case["codes"])
        codes[layer] = _codes(x * _two(-e)[..., None, None], case["codes"])
        scales[layer] = _two(e).transpose(1, 2)
    return buf, codes, scales


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
    buf, codes, scales = _cache(case, blocks, g)

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
    st = {"op": case["op"], "kind": case["codes"], "H": H, "Hkv": Hkv, "D": D, "layer": L - 1, "codes": codes, "scales": scales, "buf": buf, "nodes": dev(nodes), "seq": seq, "index": index, "N": N}
    st |= {"block": tab[seq, slot // BLOCK], "slot": slot % BLOCK, "out_type": TYPES.get(case.get("out"))}
    # rows that are read back: whole sequences, or from the page on that holds the first node
    first = [0 if case["op"] == "read" else c // BLOCK * BLOCK for c in ctx]
    rows = [(s, j) for s in range(S) for j in range(first[s], ctx[s] + counts[s])]
    row = dev(np.array(rows, dtype=np.int64))
    st["row_block"], st["row_slot"] = tab[row[:, 0], row[:, 1] // BLOCK], row[:, 1] % BLOCK
    # the pages that the nodes lie in
    pages = [(s, p) for s in range(S) for p in range(ctx[s] // BLOCK, need[s])]
    page = dev(np.array(pages, dtype=np.int64))
    number = {p: i for i, p in enumerate(pages)}
    st["page_seq"], st["page_at"], st["page_block"] = page[:, 0], page[:, 1] * BLOCK, tab[page[:, 0], page[:, 1]]
    st["page_live"] = (ctx_t[page[:, 0]] - page[:, 1] * BLOCK).clamp(min=0)  # slots of earlier tokens
    st["page_of"] = dev(np.array([number[s, (ctx[s] + i) // BLOCK] for s in range(S) for i in range(counts[s])], dtype=np.int64))

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
        key = torch.arange(longest, device="cuda")
        st["key_block"], st["key_slot"] = tab[:, key // BLOCK], key % BLOCK
        rel = key[None] - ctx_t[:, None]  # [S, keys]: negative for cached tokens, else the node's number
        seen = torch.gather(dev(sees), 2, rel.clamp(0, T - 1)[:, None].expand(S, T, longest)) & (rel < T)[:, None]
        st["sees"] = torch.where(rel[:, None] < 0, True, seen)
    elif case["op"] == "commit":
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
        pool = KvPool(shape, dec.DEC_BF16_F16KV, blocks, max_positions=40960, slabs=buf, kv_type=dec.DEC_T_I8 if case["codes"] == "i8" else dec.DEC_T_E4M3)
        pool.alloc(blocks)
        st["trees"] = DraftTrees(pool, max_seqs=S, max_tokens=N, max_blocks=max(need))
        st["trees"].set(ctx, parents, tables)
        st["all"], st["pages"] = dec.DEC_READ_ALL, dec.DEC_READ_PAGES
        if case["op"] == "append":
            kinds = {"none": dec.DEC_ROPE_PLAIN, "linear": dec.DEC_ROPE_LINEAR, "yarn": dec.DEC_ROPE_YARN, "bands": dec.DEC_ROPE_BANDS}
            more = {"yarn": {"low": 1.0, "high": 32.0, "attn_factor": 0.1 * math.log(4.0) + 1.0}, "bands": {"low": 1.0, "high": 4.0}}.get(case["scaling"], {})
            st["rope"] = RopeTable(case["rot"], longest, base=1e6, layout=dec.DEC_ROPE_HALF if st["half"] else dec.DEC_ROPE_INTERLEAVED, scaling=kinds[case["scaling"]],
                                   factor=4.0, orig_positions=4096, **more)
    return st


# ---- one pass -------------------------------------------------------------------------------------------------


def _exponent(amax, kind):
    """The smallest e of -40 .. 40 with amax <= Q 2^e: 127 = 0.9921875 2^7, 448 = 0.875 2^9."""
    f, x = torch.frexp(amax)
    e = x - torch.where(f <= 127 / 128, 7, 6) if kind == "i8" else x - torch.where(f <= 0.875, 9, 8)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX).float()


def _two(e):
    """2^e of whole e of -126 .. 127, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _log2(scale):
    """e of 2^e."""
    return (torch.frexp(scale)[1] - 1).float()


def _codes(y, kind):
    """The 8 bits of numbers that are already divided by their scale."""
    return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8) if kind == "i8" else y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _numbers(codes, kind):
    return codes.view(torch.int8).float() if kind == "i8" else codes.view(torch.float8_e4m3fn).float()


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


def _read(st, layers):
    """Rows of the cache as the numbers they stand for: keys and values [layers, rows, KV heads, D]."""
    at, slot = st["row_block"], st["row_slot"]
    x = st["codes"][layers][:, at, :, :, slot]  # [rows, layers, 2, KV heads, D]
    x = _numbers(x, st["kind"]) * st["scales"][layers][:, at].permute(1, 0, 3, 2)[..., None]
    x = x.to(st["out_type"] or torch.bfloat16).permute(2, 1, 0, 3, 4)
    return x[0].contiguous(), x[1].contiguous()


def _append(st):
    codes, scales, layer, kind = st["codes"][st["layer"]], st["scales"][st["layer"]], st["layer"], st["kind"]
    q = _rotated(st["q"], st["q_norm"], st).to(st["q_type"])
    kv = torch.stack([_rotated(st["k"], st["k_norm"], st), st["v"].float()], 1)  # [nodes, 2, KV heads, D]
    amax = kv.abs().amax(-1)
    block, live, of = st["page_block"], st["page_live"], st["page_of"]
    top = torch.zeros((len(block),) + amax.shape[1:], device=amax.device).scatter_reduce_(0, of[:, None, None].expand_as(amax), amax, "amax")
    was = _log2(scales[block]).transpose(1, 2)  # [pages, 2, KV heads]
    e = torch.maximum(_exponent(top, kind), torch.where(live[:, None, None] > 0, was, E_MIN))
    old = codes[block]
    again = _codes(_numbers(old, kind) * _two((was - e).clamp(max=0))[..., None, None], kind)
    codes[block] = torch.where(torch.arange(BLOCK, device=live.device)[:, None] < live[:, None, None, None, None], again, old)
    scales[block] = _two(e).transpose(1, 2)
    codes[st["block"], :, :, st["slot"]] = _codes(kv * _two(-e[of])[..., None], kind)
    k, v = _read(st, slice(layer, layer + 1))
    return {"q": q, "k": k[0], "v": v[0]}


def _attend(st):
    H, Hkv, D = st["H"], st["Hkv"], st["D"]
    layer = st["layer"]
    kv = _numbers(st["codes"][layer][st["key_block"], :, :, st["key_slot"]], st["kind"])  # [S, keys, 2, Hkv, D]
    kv *= st["scales"][layer][st["key_block"]].transpose(2, 3)[..., None]
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
    nodes, up, ctx, tab, codes, scales, kind = (st[k] for k in ("nodes", "up", "ctx", "tab", "codes", "scales", "kind"))
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
    # each slot of the pages: its node's number, where that comes from, whether it holds something afterwards
    seq, block = st["page_seq"], st["page_block"]
    to = st["page_at"][:, None] + torch.arange(BLOCK, device=up.device) - ctx[seq][:, None]  # [pages, 16]
    good_to = (to >= 0) & (to < n[seq][:, None])
    frm = torch.where(good_to, path[seq[:, None], to.clamp(0, T - 1)], to)
    live, moved = (to < 0) | good_to, good_to & (frm != to)
    pos = torch.where(live, ctx[seq][:, None] + frm, st["page_at"][:, None])
    src_block, src_slot = tab[seq[:, None], pos // BLOCK], pos % BLOCK
    was = _log2(scales).permute(1, 0, 3, 2)  # [blocks, layers, 2, KV heads]
    x = _numbers(codes[:, src_block, :, :, src_slot], kind) * _two(was[src_block])[..., None]  # [pages, 16, layers, 2, KV heads, D]
    top = torch.where(moved[:, :, None, None, None], x.abs().amax(-1), 0.0).amax(1)
    e = torch.maximum(was[block], _exponent(top, kind))  # [pages, layers, 2, KV heads]
    new = _codes(x * _two(-e)[:, None, ..., None], kind)
    old = codes[:, block].permute(1, 4, 0, 2, 3, 5)
    codes[:, block] = torch.where(live[:, :, None, None, None, None], new, old).permute(2, 0, 3, 4, 1, 5)
    scales[:, block] = _two(e).permute(1, 0, 3, 2)
    last = torch.gather(path, 1, (n - 1)[:, None])
    k, v = _read(st, slice(None))
    return {"accepted": n.int(), "path": torch.where(good, path, -1)[nodes < st["N"]].int(), "next": torch.gather(target, 1, last)[:, 0], "k": k, "v": v}


def run(st):
    if own:
        trees = st["trees"]
        if st["op"] == "append":  # the step's keys and values go in, and the pages that they changed come back
            q = trees.append(st["layer"], st["q"], st["k"], st["v"], rope=st["rope"], q_norm=st["q_norm"], k_norm=st["k_norm"], q_type=st["q_type"])
            k, v = trees.read(st["layer"], part=st["pages"])
            return {"q": q, "k": k, "v": v}
        if st["op"] == "attend":
            return trees.attend(st["layer"], st["q"], out_type=st["out_type"])
        if st["op"] == "read":
            k, v = trees.read(0, layers=len(st["codes"]), part=st["all"], out_type=st["out_type"])
            return {"k": k, "v": v}
        accepted, path, after = trees.commit(st["draft"], st["target"])
        k, v = trees.read(0, layers=len(st["codes"]), part=st["pages"], out_type=st["out_type"])
        return {"accepted": accepted, "path": path, "next": after, "k": k, "v": v}
    if st["op"] == "read":
        k, v = _read(st, slice(None))
        return {"k": k, "v": v}
    return {"append": _append, "attend": _attend, "commit": _commit}[st["op"]](st)


# ---- what a pass cannot do without ----------------------------------------------------------------------------


def work(case):
    ctx, counts = _sizes(case)
    H, Hkv, D, N, L = case["heads"], case["kv_heads"], case["head_dim"], sum(counts), _layers(case)
    pages = sum((c + n + BLOCK - 1) // BLOCK - c // BLOCK for c, n in zip(ctx, counts))
    back = sum(c % BLOCK + n for c, n in zip(ctx, counts))  # rows that are read back behind an append or a commit
    if case["op"] == "append":
        width = SIZE[case["in"]]
        moved = N * D * (H * (width + SIZE[case["q_out"]]) + 2 * Hkv * (width + 1)) + N * case["rot"] * 4 + back * 2 * Hkv * D * 2 + (back - N) * 2 * Hkv * D + pages * Hkv * 8
        return {"bytes": moved, "flops": N * (H + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0)) + 4 * N * Hkv * D}
    keys = sum(c + n for c, n in zip(ctx, counts))
    if case["op"] == "attend":
        scales = 8 * Hkv * sum((c + n + BLOCK - 1) // BLOCK for c, n in zip(ctx, counts))
        return {"bytes": 2 * keys * Hkv * D + scales + N * H * D * (SIZE[case["in"]] + SIZE[case["out"]]), "flops": sum(4 * D * H * n * (c + n / 2) for c, n in zip(ctx, counts))}
    if case["op"] == "read":
        return {"bytes": keys * L * 2 * Hkv * D * (1 + SIZE[case["out"]]), "flops": keys * L * 2 * Hkv * D}
    rows = sum(max(min(case["accept"], n) - 1, 0) for n in counts)
    rows = 0 if case["tree"] == "chain" else rows  # a chain's accepted nodes are in place
    return {"bytes": 4 * rows * L * Hkv * D + 16 * N + back * L * 2 * Hkv * D * (1 + SIZE[case["out"]]), "flops": back * L * 2 * Hkv * D}


# ---- the definition, in 64 bits --------------------------------------------------------------------------------


class _Pages:
    """A cache as what it stands for, in 64 bits: page by page, written row by row."""

    def __init__(self, st):
        self.kind, self.top = st["kind"], 127.0 if st["kind"] == "i8" else 448.0
        c = st["codes"].view(torch.int8).double() if st["kind"] == "i8" else st["codes"].view(torch.float8_e4m3fn).double()
        self.scale = st["scales"].double().permute(0, 1, 3, 2).clone()  # [layers, blocks, 2, KV heads]
        self.value = c * self.scale[..., None, None]  # [layers, blocks, 2, KV heads, 16, D]

    def rounded(self, x, scale):
        y = x / scale
        if self.kind == "i8":
            y = torch.round(y)
        else:  # three bits behind the leading one, none below 2^-9
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = torch.round(y / step) * step
        return y.clamp(-self.top, self.top) * scale

    def write(self, layers, block, rows, slots, keep, begun):
        """Rows [n, layers, 2, KV heads, D] to the slots of a block whose slots `keep` hold earlier tokens; begun: nothing else counts for its scale."""
        need = rows.abs().amax((0, -1))
        scale = torch.full_like(need, 2.0 ** E_MIN)
        while bool((need > self.top * scale).logical_and(scale < 2.0 ** E_MAX).any()):
            scale = torch.where((need > self.top * scale) & (scale < 2.0 ** E_MAX), scale * 2, scale)
        was = self.scale[layers, block]
        if not begun:
            scale = torch.maximum(scale, was)
        for j in keep:
            row = self.value[layers, block][:, :, :, j]
            self.value[layers, block, :, :, j] = torch.where((scale > was)[..., None], self.rounded(row, scale[..., None]), row)
        for j in range(BLOCK):
            if j not in keep and j not in slots:  # what a slot without a token holds are its bits
                self.value[layers, block, :, :, j] *= (scale / was)[..., None]
        for row, j in zip(rows, slots):
            self.value[layers, block, :, :, j] = self.rounded(row, scale[..., None])
        self.scale[layers, block] = scale

    def rows(self, layers, st):
        x = self.value[layers][:, st["row_block"], :, :, st["row_slot"]].permute(2, 1, 0, 3, 4)
        return x[0], x[1]


def exact(case, seed):
    st = prepare(case, seed)
    ctx, counts = _sizes(case)
    H, Hkv, D, layer = st["H"], st["Hkv"], st["D"], st["layer"]
    if case["op"] == "read":
        k, v = _Pages(st).rows(slice(None), st)
        return {"k": k, "v": v}
    if case["op"] == "append":
        pages = _Pages(st)
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

        kv = torch.stack([formed(st["k"], st["k_norm"]), st["v"].double()], 1)[:, None]  # [nodes, 1, 2, KV heads, D]
        block, slot = st["block"].tolist(), st["slot"].tolist()
        b = 0
        for c, n in zip(ctx, counts):
            i = 0
            while i < n:
                m = min(n - i, BLOCK - (c + i) % BLOCK)
                held = list(range((c + i) % BLOCK)) if i == 0 else []
                pages.write(slice(layer, layer + 1), block[b + i], kv[b + i:b + i + m], slot[b + i:b + i + m], held, not held)
                i += m
            b += n
        k, v = pages.rows(slice(layer, layer + 1), st)
        return {"q": formed(st["q"], st["q_norm"]), "k": k[0], "v": v[0]}
    if case["op"] == "attend":
        if sum(4 * D * H * n * (c + n) for c, n in zip(ctx, counts)) > 4e11:
            return None
        pages = _Pages(st)
        out = torch.empty((st["N"], H, D), dtype=torch.float64, device="cuda")
        b = 0
        for s, (c, n) in enumerate(zip(ctx, counts)):
            rows = pages.value[layer][st["key_block"][s, :c + n], :, :, st["key_slot"][:c + n]]  # [keys, 2, Hkv, D]
            for h in range(H):
                kv = rows[:, :, h * Hkv // H]
                score = st["q"][b:b + n, h].double() @ kv[:, 0].T * D ** -0.5
                weight = torch.softmax(torch.where(st["sees"][s, :n, :c + n], score, -math.inf), dim=-1)
                out[b:b + n, h] = weight @ kv[:, 1]
            b += n
        return out.flatten(1)
    # commit: the walk and the move, node by node
    pages, b = _Pages(st), 0
    draft, target, up, tab = (st[k].tolist() for k in ("draft", "target", "up", "tab"))
    accepted, path, after = [], [], []
    every = slice(None)
    for s, n in enumerate(counts):
        at, way = 0, [0]
        while True:
            to = [i for i in range(n) if up[s][i] == at and draft[b + i] == target[b + at]]
            if not to:
                break
            at = to[0]
            way.append(at)
        for p in range(ctx[s] // BLOCK, (ctx[s] + len(way) + BLOCK - 1) // BLOCK):
            mine = [(i, w) for i, w in enumerate(way) if (ctx[s] + i) // BLOCK == p]
            going = [(i, w) for i, w in mine if i != w]
            if going:
                rows = torch.stack([pages.value[:, tab[s][(ctx[s] + w) // BLOCK], :, :, (ctx[s] + w) % BLOCK] for _, w in going])
                stay = list(range(max(0, min(BLOCK, ctx[s] - p * BLOCK)))) + [(ctx[s] + i) % BLOCK for i, w in mine if i == w]
                pages.write(every, tab[s][p], rows, [(ctx[s] + i) % BLOCK for i, _ in going], stay, False)
        accepted.append(len(way))
        path += way + [-1] * (n - len(way))
        after.append(target[b + at])
        b += n
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = pages.rows(every, st)
    return {"accepted": whole(accepted), "path": whole(path), "next": whole(after), "k": k, "v": v}
