"""Draft trees over the paged cache on the GPU: append, attention and commit
against plain implementations in 64 bits, and the calls that could go wrong:
empty and ragged trees, pages that end anywhere, values in slots nobody sees,
padding, strides, types, captured and replayed calls, two plans at once, a
pool past 2^31 elements."""

import ctypes as C
import math
import random

import pytest

torch = pytest.importorskip("torch")

from decoder_qwen3_step_gb300 import dec  # noqa: E402
from decoder_qwen3_step_gb300.trees import DraftTrees, KvPool, RopeTable  # noqa: E402

pytestmark = pytest.mark.gpu

PAD = dec.DEC_TREE_PAD
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SHAPES = {"4:2x32": (4, 2, 32), "8:4x64": (8, 4, 64), "16:8x128": (16, 8, 128), "5:5x64": (5, 5, 64), "12:3x32": (12, 3, 32), "8:2x128": (8, 2, 128)}
CACHE = {"f32": torch.float32, "f16": torch.float16}


class Setup:
    """A pool of random K/V, pages in random order, and a plan of the given trees."""

    def __init__(self, shape, cache, ctx, parents, layers=2, seed=0, spare=3, max_tokens=None, extra_blocks=0):
        self.H, self.Hkv, self.D = SHAPES[shape]
        self.cache, self.layers = CACHE[cache], layers
        rng = random.Random(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.ctx, self.parents = list(ctx), [list(range(-1, p - 1)) if isinstance(p, int) else list(p) for p in parents]
        need = [(c + len(p) + 15) // 16 for c, p in zip(self.ctx, self.parents)]
        self.blocks = sum(need) + spare + extra_blocks
        self.shape = {"vocab": 512, "d_model": 64, "n_layers": layers, "n_heads": self.H, "n_kv_heads": self.Hkv, "head_dim": self.D, "ff_hidden": 64}
        self.slab = torch.randn((layers, self.blocks, 2, self.Hkv, 16, self.D), generator=self.g).to(self.cache).cuda()
        self.pool = KvPool(self.shape, dec.DEC_FP32 if cache == "f32" else dec.DEC_BF16_F16KV, self.blocks, max_positions=40960, slabs=self.slab)
        ids = self.pool.alloc(self.blocks)
        rng.shuffle(ids)
        self.tables = [[ids.pop() for _ in range(n)] for n in need]
        self.N = sum(len(p) for p in self.parents)
        self.trees = DraftTrees(self.pool, max(len(self.ctx), 1), max_tokens or self.N, max(need + [1]) + 2)
        self.trees.set(self.ctx, self.parents, self.tables)

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g).cuda()

    def where(self, s, slot):
        return self.tables[s][slot // 16], slot % 16

    def nodes(self):
        """(node, sequence, number in it, slot, position or None for padding) of every node."""
        n = 0
        for s, tree in enumerate(self.parents):
            depth = []
            for i, p in enumerate(tree):
                depth.append(None if p == PAD else 0 if p < 0 else depth[p] + 1)
                yield n, s, i, self.ctx[s] + i, None if p == PAD else self.ctx[s] + depth[i]
                n += 1

    def seen(self, s, i):
        """Slots that node i of sequence s sees."""
        if self.parents[s][i] == PAD:
            return []
        way, at = [], i
        while at >= 0:
            way.append(self.ctx[s] + at)
            at = self.parents[s][at]
        return list(range(self.ctx[s])) + sorted(way)

    def kv(self, layer, s, slots):
        b = torch.tensor([self.where(s, x)[0] for x in slots], dtype=torch.long, device="cuda")
        r = torch.tensor([x % 16 for x in slots], dtype=torch.long, device="cuda")
        rows = self.slab[layer][b, :, :, r]  # [slots, 2, Hkv, D]
        return rows[:, 0].double(), rows[:, 1].double()

    def close(self):
        torch.cuda.synchronize()
        assert self.trees.status() == 0
        self.trees.close()
        self.pool.close()


def reference(w, layer, q, only=None):
    """The formula in 64 bits, node by node: outputs [N, H, D], and how far a right kernel may be off them."""
    out = torch.zeros((w.N, w.H, w.D), dtype=torch.float64, device="cuda")
    tol = torch.zeros((w.N, w.H, 1), dtype=torch.float64, device="cuda")
    G = w.H // w.Hkv
    for n, s, i, slot, pos in w.nodes():
        if pos is None or (only is not None and n not in only):
            continue
        k, v = w.kv(layer, s, w.seen(s, i))
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        qn = q[n].double()
        sc = torch.einsum("hd,khd->hk", qn, k) / math.sqrt(w.D)
        size = torch.einsum("hd,khd->hk", qn.abs(), k.abs()) / math.sqrt(w.D)  # what the score's roundings are relative to
        p = torch.softmax(sc, -1)
        out[n] = torch.einsum("hk,khd->hd", p, v)
        spread = torch.einsum("hk,khd->hd", p, v.abs()).amax(-1)
        # a score off by e changes its weight by a factor within exp(+-e), the sum likewise; fp32: products and
        # partial sums, D + 4 half steps of their size, the exponential's argument and result 4 more; f16
        # queries and weights: half a step each; a sum over the keys rounds like sqrt(keys) half steps or less, 64 cover it
        worst = (p * size).sum(-1) + size.amax(-1)
        fp32 = (w.D + 8) * 2.0 ** -24 * worst + (64 + 8) * 2.0 ** -24
        f16 = 0.0 if w.cache == torch.float32 else 2.0 ** -11 * worst + 2 * 2.0 ** -11
        tol[n, :, 0] = (fp32 + f16) * spread * 1.01 + 1e-30
    return out, tol


def check(w, out, layer, q, only=None):
    ref, tol = reference(w, layer, q, only)
    got = out.view(w.N, w.H, w.D).double()
    if only is not None:
        got, ref, tol = got[only], ref[only], tol[only]
    off = (got - ref).abs()
    allowed = tol + HALF_STEP[out.dtype] * (ref.abs() + tol)
    assert bool(torch.isfinite(got).all())
    bad = off > allowed
    assert not bool(bad.any()), (int(bad.sum()), float((off / allowed).max()), bad.nonzero()[:4].tolist())
    # and as a whole the roundings do not pull one way: two half steps of the output type cover them
    if w.cache == torch.float32:
        assert float(off.norm()) <= 2e-6 * float(ref.norm()) + 1e-12
    else:
        assert float(off.norm()) <= 2 * 2.0 ** -9 * float(ref.norm()) + 1e-12


def random_tree(n, seed):
    rng = random.Random(seed)
    return [-1] + [rng.randint(-1 if rng.random() < 0.1 else 0, i - 1) for i in range(1, n)]


BATCHES = {
    "one node, nothing cached": ([0], [1]),
    "one node, one cached": ([1], [1]),
    "page borders": ([15, 16, 17, 31, 47, 48], [1, 1, 1, 2, 1, 16]),
    "tile borders": ([62, 63, 64, 65, 127, 128], [2, 1, 1, 3, 2, [-1, 0, 0]]),
    "siblings of the root only": ([20], [[-1] * 40]),
    "ragged with empty sequences": ([5, 100, 0, 77], [0, random_tree(9, 1), random_tree(33, 2), 0]),
    "widest chain": ([300], [256]),
    "widest tree": ([130, 3], [random_tree(256, 3), random_tree(131, 4)]),
    "many sequences": ([7 * i for i in range(33)], [random_tree(1 + (i * 11) % 17, i) for i in range(33)]),
    "long cache": ([5003], [random_tree(21, 5)]),
    "padding": ([40, 9], [[-1, PAD, 0, 0, PAD, 2, PAD], [PAD, PAD]]),
}


@pytest.mark.parametrize("cache", ["f16", "f32"])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_attention_is_the_formula(batch, shape, cache):
    ctx, parents = BATCHES[batch]
    w = Setup(shape, cache, ctx, parents, seed=len(batch))
    q = w.rand(w.N, w.H, w.D)
    out = torch.full((w.N, w.H * w.D), float("nan"), dtype=torch.float32 if cache == "f32" else torch.bfloat16, device="cuda")
    w.trees.attend(1, q, out=out)
    few = sorted(random.Random(1).sample(range(w.N), min(w.N, 60)))
    check(w, out, 1, q, few)
    pads = [n for n, _, _, _, pos in w.nodes() if pos is None]
    assert not bool(out[pads].any())
    w.close()


@pytest.mark.parametrize("cache", ["f16", "f32"])
@pytest.mark.parametrize("shape", ["8:4x64", "16:8x128", "4:2x32"])
def test_values_in_slots_that_a_node_does_not_see_change_nothing(shape, cache):
    ctx, parents = [37, 70, 0], [random_tree(23, 1), [-1, 0, 0, 1, 1, 2], random_tree(90, 2)]
    w = Setup(shape, cache, ctx, parents, seed=9)
    q = w.rand(w.N, w.H, w.D)
    clean = w.trees.attend(0, q).clone()
    # everything that belongs to no slot of any sequence: the rest of the last pages, the other pages, the other layer
    mask = torch.ones(w.slab.shape[1], 16, dtype=torch.bool, device="cuda")
    for s in range(3):
        for slot in range(w.ctx[s] + len(w.parents[s])):
            b, r = w.where(s, slot)
            mask[b, r] = False
    w.slab[0].permute(0, 3, 1, 2, 4)[mask] = float("nan")
    w.slab[1] = float("inf")
    assert torch.equal(w.trees.attend(0, q), clean)
    # one node's key and value are not finite: its descendants' rows are not either, nobody else's change
    for value in (float("nan"), float("inf"), -float("inf")):
        for s, i in ((0, 3), (1, 2), (2, 40)):
            b, r = w.where(s, w.ctx[s] + i)
            keep = w.slab[0, b, :, :, r].clone()
            n0 = sum(len(p) for p in w.parents[:s])
            below = torch.tensor([n0 + j for j in range(len(w.parents[s])) if w.ctx[s] + i in w.seen(s, j)], device="cuda")
            rest = torch.ones(w.N, dtype=torch.bool, device="cuda")
            rest[below] = False
            for kv in (0, 1):
                w.slab[0, b, kv, :, r] = value
                got = w.trees.attend(0, q)
                assert torch.equal(got[rest], clean[rest]), (value, s, i, kv)
                if kv == 1 or math.isnan(value):
                    assert not bool(torch.isfinite(got[below]).any()), (value, s, i, kv)
                w.slab[0, b, :, :, r] = keep
    assert torch.equal(w.trees.attend(0, q), clean)
    w.close()


@pytest.mark.parametrize("cache, seqs, nodes, ctx", [("f32", 1, 20, 3000), ("f16", 1, 6, 3000), ("f16", 30, 7, 900), ("f16", 2, 60, 3000),
                                                     ("f16", 30, 50, 900), ("f16", 2, 250, 1500), ("f16", 10, 200, 900)])
def test_values_that_are_not_finite_in_units_that_share_their_keys(cache, seqs, nodes, ctx):
    """Contexts that several CTAs divide, their parts put together by a second kernel or by one of them."""
    w = Setup("16:8x128", cache, [ctx + 3 * i for i in range(seqs)], [random_tree(nodes, i) for i in range(seqs)], seed=4)
    q = w.rand(w.N, w.H, w.D)
    clean = w.trees.attend(0, q).clone()
    check(w, clean, 0, q, sorted(random.Random(3).sample(range(w.N), min(w.N, 20))))
    for value in (float("nan"), float("inf")):
        for s, i in ((0, 2), (seqs - 1, nodes // 2)):
            b, r = w.where(s, w.ctx[s] + i)
            keep = w.slab[0, b, 1, :, r].clone()
            below = torch.tensor([nodes * s + j for j in range(nodes) if w.ctx[s] + i in w.seen(s, j)], device="cuda")
            rest = torch.ones(w.N, dtype=torch.bool, device="cuda")
            rest[below] = False
            w.slab[0, b, 1, :, r] = value
            got = w.trees.attend(0, q)
            assert torch.equal(got[rest], clean[rest]), (value, s, i)
            assert not bool(torch.isfinite(got[below]).any()), (value, s, i)
            w.slab[0, b, 1, :, r] = keep
    assert torch.equal(w.trees.attend(0, q), clean)
    w.close()


@pytest.mark.parametrize("cache", ["f16", "f32"])
@pytest.mark.parametrize("in_type", [torch.float32, torch.bfloat16, torch.float16])
def test_types_strides_and_rows_behind_the_last(in_type, cache):
    w = Setup("16:8x128", cache, [50, 3], [random_tree(19, 3), 7], seed=2)
    wide = w.rand(w.N + 3, (w.H + 2 * w.Hkv) * w.D + 4).to(in_type)
    q = wide[: w.N, 4: 4 + w.H * w.D]  # rows of a wider buffer
    types = [torch.float32, torch.float16, torch.bfloat16] if cache == "f32" else [torch.float16, torch.bfloat16]
    for t in types:
        buf = torch.full((w.N + 2, w.H * w.D + 8), 7.0, dtype=t, device="cuda")
        out = buf[: w.N, 4: 4 + w.H * w.D]
        w.trees.attend(1, q, out=out)
        got = out.contiguous()
        ref, tol = reference(w, 1, q.view(w.N, w.H, w.D) if q.is_contiguous() else q.reshape(w.N, w.H, w.D))
        off = (got.view(w.N, w.H, w.D).double() - ref).abs()
        assert bool((off <= tol + HALF_STEP[t] * (ref.abs() + tol)).all())
        out.fill_(7.0)
        assert bool((buf == 7.0).all())
    w.close()


@pytest.mark.parametrize("scale", [1e30, 1e-30, 70000.0, 0.0])
def test_queries_of_any_magnitude(scale):
    w = Setup("8:4x64", "f16", [100], [random_tree(20, 3)], seed=4)
    q = w.rand(w.N, w.H, w.D)
    out = w.trees.attend(0, q * scale).view(w.N, w.H, w.D).double()
    G = w.H // w.Hkv
    for n, s, i, slot, pos in w.nodes():
        k, v = (x.repeat_interleave(G, 1) for x in w.kv(0, s, w.seen(s, i)))
        sc = torch.einsum("hd,khd->hk", q[n].double() * scale, k) / 8.0
        top = sc.topk(2, -1).values
        p = torch.softmax(sc, -1)
        ref = torch.einsum("hk,khd->hd", p, v)
        # huge scores: one key takes all, where its lead is above the rounding of the scores
        size = torch.einsum("hd,khd->hk", q[n].double().abs() * scale, k.abs()).amax(-1) / 8.0
        sure = (top[:, 0] - top[:, 1] > 4 * 2.0 ** -11 * size + 20) if scale > 1 else torch.ones(w.H, dtype=torch.bool, device="cuda")
        tol = (2 * 2.0 ** -11 + 2.0 ** -8) * v.abs().amax(0) + 1e-4
        assert bool(((out[n] - ref).abs() <= tol)[sure].all()), (scale, n)
    assert bool(torch.isfinite(out).all())
    w.close()


def test_a_head_row_past_two_to_the_31():
    """The pool's last layer starts past 2^31 elements."""
    w = Setup("16:8x128", "f16", [33], [random_tree(12, 3)], layers=28, seed=1, extra_blocks=2600)
    assert w.slab.numel() > 2 ** 31
    q, k, v = w.rand(w.N, w.H, w.D), w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    w.trees.append(27, None, k, v)
    for n, s, i, slot, pos in w.nodes():
        b, r = w.where(s, slot)
        assert torch.equal(w.slab[27, b, 0, :, r], k[n].half()) and torch.equal(w.slab[27, b, 1, :, r], v[n].half())
    check(w, w.trees.attend(27, q), 27, q)
    w.close()


# ---- append -----------------------------------------------------------------------------------------------------


def frequencies(rot, base, scaling, factor, orig, low, high):
    f = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if scaling == dec.DEC_ROPE_LINEAR:
        return [x / factor for x in f]
    if scaling == dec.DEC_ROPE_YARN:
        index = lambda turns: rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        a, b = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
        g = [min(max((j - a) / max(b - a, 0.001), 0.0), 1.0) for j in range(rot // 2)]
        return [x * (1 - y) + x / factor * y for x, y in zip(f, g)]
    if scaling == dec.DEC_ROPE_BANDS:
        g = [min(max((orig * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        return [x * y + x / factor * (1 - y) for x, y in zip(f, g)]
    return f


SCALINGS = {"plain": (dec.DEC_ROPE_PLAIN, {}), "linear": (dec.DEC_ROPE_LINEAR, {"factor": 8.0}),
            "yarn": (dec.DEC_ROPE_YARN, {"factor": 4.0, "orig_positions": 2048, "low": 1.0, "high": 32.0, "attn_factor": 1.138}),
            "bands": (dec.DEC_ROPE_BANDS, {"factor": 8.0, "orig_positions": 8192, "low": 1.0, "high": 4.0})}


def formed(x, gain, pos, rot, layout, freq, mult):
    """RMSNorm and rotation in 64 bits."""
    x = x.double()
    if gain is not None:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
    if not rot:
        return x
    angle = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    c, s = angle.cos() * mult, angle.sin() * mult
    y = x.clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == dec.DEC_ROPE_HALF else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


@pytest.mark.parametrize("shape, rot", [("4:2x32", 8), ("4:2x32", 32), ("8:4x64", 48), ("16:8x128", 128), ("16:8x128", 72), ("5:5x64", 64), ("12:3x32", 24)])
@pytest.mark.parametrize("layout", [dec.DEC_ROPE_HALF, dec.DEC_ROPE_INTERLEAVED])
@pytest.mark.parametrize("scaling", list(SCALINGS))
def test_append_is_the_formula(shape, rot, layout, scaling):
    kind, more = SCALINGS[scaling]
    number = rot + 2 * layout + len(scaling)
    cache = ["f16", "f32"][number % 2]
    in_type = [torch.float32, torch.bfloat16, torch.float16][number % 3]
    q_type = [torch.float32, torch.bfloat16][number % 2]
    norm = scaling != "linear"
    # one sequence far out, where a 32-bit angle would be wrong
    w = Setup(shape, cache, [0, 17, 31, 38000 if shape == "4:2x32" else 900], [random_tree(20, 1), 3, [-1, PAD, 0], 2], seed=number)
    rope = RopeTable(rot, 40000, base=1e6, layout=layout, scaling=kind, **more)
    raw = w.rand(w.N, (w.H + 2 * w.Hkv) * w.D).to(in_type)
    q, k, v = (x.view(w.N, -1, w.D) for x in raw.split([w.H * w.D, w.Hkv * w.D, w.Hkv * w.D], 1))
    gq, gk = (1 + 0.1 * w.rand(w.D), 1 + 0.1 * w.rand(w.D)) if norm else (None, None)
    before = w.slab.clone()
    got = w.trees.append(1, q, k, v, rope=rope, q_norm=gq, k_norm=gk, q_type=q_type)
    where = list(w.nodes())
    pos = torch.tensor([p or 0 for *_, p in where], device="cuda")
    live = torch.tensor([p is not None for *_, p in where], device="cuda")
    freq = frequencies(rot, 1e6, kind, more.get("factor"), more.get("orig_positions"), more.get("low"), more.get("high"))
    mult = more.get("attn_factor", 1.0)

    def near(a, x, gain, name):
        ref = formed(x, gain, pos, rot, layout, freq, mult)[live]
        # the table's rounding, two products and their sum; with a norm the D squares' sum and five operations more
        size = ref.abs() + (formed(x, gain, pos, 0, 0, freq, 1.0).abs().amax(-1, keepdim=True) * 2)[live]
        off = (a.double() - ref).abs()
        allowed = (4 + (w.D / 2 + 6 if gain is not None else 0)) * 2.0 ** -24 * size + HALF_STEP[a.dtype] * ref.abs() * 1.001 + 2.0 ** -25 * (a.dtype == torch.float16)
        assert bool((off <= allowed).all()), (name, float((off / allowed).max()))

    near(got[live], q, gq, "q")
    assert not bool(got[~live].any())
    blocks = torch.tensor([w.where(s, slot)[0] for _, s, _, slot, _ in where], device="cuda")[live]
    rows = torch.tensor([slot % 16 for _, _, _, slot, _ in where], device="cuda")[live]
    near(w.slab[1][blocks, 0, :, rows], k, gk, "k")
    assert torch.equal(w.slab[1][blocks, 1, :, rows], v[live].to(w.cache))
    # nothing else moved
    w.slab[1].index_put_((blocks, torch.zeros_like(blocks)), before[1][blocks, 0])
    w.slab[1].index_put_((blocks, torch.ones_like(blocks)), before[1][blocks, 1])
    rest = torch.ones(w.slab.shape[1], 16, dtype=torch.bool, device="cuda")
    rest[blocks, rows] = False
    assert torch.equal(w.slab[0], before[0])
    assert torch.equal(w.slab[1].permute(0, 3, 1, 2, 4)[rest], before[1].permute(0, 3, 1, 2, 4)[rest])
    w.close()


@pytest.mark.parametrize("cache", ["f16", "f32"])
def test_append_of_parts_in_place_and_without_rotation(cache):
    w = Setup("8:4x64", cache, [5], [random_tree(9, 1)], seed=1)
    q, k, v = w.rand(w.N, w.H, w.D), w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    before = w.slab.clone()
    assert torch.equal(w.trees.append(0, q, None, None), q)  # queries alone, nothing to do to them
    assert torch.equal(w.slab, before)
    rope = RopeTable(64, 100)
    want = w.trees.append(0, q, None, None, rope=rope)
    inplace = q.clone()
    assert w.trees.append(0, inplace, None, None, rope=rope, out=inplace) is inplace and torch.equal(inplace, want)
    assert w.trees.append(1, None, k, v) is None
    for n, s, i, slot, pos in w.nodes():
        b, r = w.where(s, slot)
        assert torch.equal(w.slab[1, b, 0, :, r], k[n].to(w.cache)) and torch.equal(w.slab[1, b, 1, :, r], v[n].to(w.cache))
    big = torch.full_like(k, 1e6)  # past f16: infinity, as the cache's own conversion
    w.trees.append(1, None, big, v)
    b, r = w.where(0, 5)
    assert torch.equal(w.slab[1, b, 0, :, r], big[0].to(w.cache))
    w.close()


def test_the_widest_append():
    w = Setup("16:8x128", "f16", [3] * 33, [256] * 33, layers=1, seed=1)
    k, v = w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    q = w.rand(w.N, w.H, w.D)
    rope = RopeTable(128, 300)
    got = w.trees.append(0, q, k, v, rope=rope)
    pos = torch.tensor([p for *_, p in w.nodes()], device="cuda")
    ref = formed(q, None, pos, 128, dec.DEC_ROPE_HALF, frequencies(128, 1e6, 0, 1, 1, 1, 1), 1.0)
    assert float((got.double() - ref).abs().max()) <= 4 * 2.0 ** -24 * 2 * float(q.abs().max())
    kk, vv = (torch.stack([w.slab[0, w.where(s, slot)[0], z, :, slot % 16] for _, s, _, slot, _ in w.nodes()]) for z in (0, 1))
    assert torch.equal(vv, v.half())
    ref = formed(k, None, pos, 128, dec.DEC_ROPE_HALF, frequencies(128, 1e6, 0, 1, 1, 1, 1), 1.0)
    assert float((kk.double() - ref).abs().max()) <= (8 * 2.0 ** -24 + 2.0 ** -11) * 2 * float(k.abs().max())
    w.close()


# ---- commit ------------------------------------------------------------------------------------------------------


def walk(parents, draft, target, prior):
    at, way = -1, []
    while True:
        want = (lambda i: True) if at < 0 and prior is None else (lambda i: draft[i] == (prior if at < 0 else target[at]))
        to = [i for i, p in enumerate(parents) if p == at and want(i)]
        if not to:
            return way
        at = to[0]
        way.append(at)


@pytest.mark.parametrize("cache", ["f16", "f32"])
@pytest.mark.parametrize("with_prior", [False, True])
@pytest.mark.parametrize("shape", ["4:2x32", "16:8x128", "5:5x64"])
def test_commit_walks_and_moves(shape, with_prior, cache):
    parents = [random_tree(30, 1), 256, [-1], random_tree(200, 2), [], [-1, 0, 0, 0, 1, 2, 3, 4, 5, 6], [-1, PAD, 0, PAD, 2], [PAD], [-1, -1, -1, 2, 2, 4], list(range(-1, 11)) + [0] * 30]
    ctx = [13, 7, 0, 30, 50, 16, 31, 4, 9, 15]
    w = Setup(shape, cache, ctx, parents, layers=3, seed=5)
    rng = random.Random(shape + cache)
    draft = [rng.randrange(3) for _ in range(w.N)]  # few tokens: many siblings agree, long ways are accepted
    target = [rng.randrange(3) for _ in range(w.N)]
    n0 = len(parents[0])
    for i in range(256):  # the chain is accepted whole
        draft[n0 + i] = i
        target[n0 + i] = i + 1
    n5 = sum(len(p) if isinstance(p, list) else p for p in parents[:5])
    draft[n5: n5 + 10] = target[n5: n5 + 10] = [1] * 10  # and here all siblings agree: 0, 1, 4, 7
    prior = [rng.randrange(3) for _ in parents]
    prior[1], prior[5] = 0, 1
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want = w.slab.clone()
    acc, path, nxt, b = [], [], [], 0
    for s, tree in enumerate(w.parents):
        d, t = draft[b: b + len(tree)], target[b: b + len(tree)]
        way = walk(tree, d, t, prior[s] if with_prior else None)
        for i, x in enumerate(way):
            (bd, rd), (bs, rs) = w.where(s, ctx[s] + i), w.where(s, ctx[s] + x)
            want[:, bd, :, :, rd] = w.slab[:, bs, :, :, rs]
        acc.append(len(way))
        path += way + [-1] * (len(tree) - len(way))
        nxt.append(t[way[-1]] if way else prior[s] if with_prior else -1)
        b += len(tree)
    a, p, x = w.trees.commit(dev(draft), dev(target), dev(prior) if with_prior else None)
    assert a.tolist() == acc and p.tolist() == path and x.tolist() == nxt
    assert acc[1] == 256 and acc[5] == 4
    # behind the accepted nodes a slot holds what it held
    assert torch.equal(w.slab, want)
    w.close()


# ---- together -----------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("cache", ["f16", "f32"])
@pytest.mark.parametrize("shape", ["8:4x64", "16:8x128"])
def test_steps_of_drafting_give_the_plain_sequence(shape, cache):
    """Three steps over two layers: trees appended and attended, paths
    committed.  What the accepted nodes computed, and the cache they leave,
    are those of the same tokens taken one by one."""
    H, Hkv, D = SHAPES[shape]
    rng, steps, room = random.Random(7), 3, 40
    a = Setup(shape, cache, [21, 60], [room, room], seed=3)  # room for all steps
    plain = a.slab.clone()
    ctx = [21, 60]
    rope = RopeTable(D, 200)
    gain = 1 + 0.1 * a.rand(D)
    vocab = 50
    table = {kind: a.rand(vocab, n * D) for kind, n in (("q", H), ("k", Hkv), ("v", Hkv))}  # a token's raw rows
    taken = [[], []]
    outs = [[], []]
    pending = [rng.randrange(vocab) for _ in range(2)]
    for step in range(steps):
        parents = [random_tree(12, 10 * step), random_tree(5, 10 * step + 1)]
        parents = [[-1] + [max(p, 0) for p in t[1:]] for t in parents]
        draft, target = [], []
        for s, tree in enumerate(parents):
            d = [rng.randrange(vocab) for _ in tree]
            d[0] = pending[s]
            t = [rng.randrange(vocab) for _ in tree]
            for i, p in enumerate(tree):  # some children are what the model chooses
                if p >= 0 and rng.random() < 0.6:
                    t[p] = d[i]
            draft += d
            target += t
        a.trees.set(ctx, parents, a.tables)
        a.ctx, a.parents, a.N = ctx, parents, len(draft)
        ids = torch.tensor(draft, device="cuda")
        per_layer = []
        for layer in range(2):
            q, k, v = (table[x][ids].view(len(draft), -1, D) for x in "qkv")
            q = a.trees.append(layer, q, k, v, rope=rope, q_norm=gain, k_norm=gain)
            per_layer.append(a.trees.attend(layer, q))
        acc, path, nxt = a.trees.commit(ids.int(), torch.tensor(target, dtype=torch.int32, device="cuda"))
        b = 0
        for s, tree in enumerate(parents):
            n = int(acc[s])
            way = path[b: b + n].tolist()
            assert n >= 1 and way[0] == 0
            taken[s] += [draft[b + i] for i in way]
            outs[s] += [[o[b + i] for o in per_layer] for i in way]
            pending[s] = int(nxt[s])
            ctx = ctx[:s] + [ctx[s] + n] + ctx[s + 1:]
            b += len(tree)
    got = a.slab.clone()
    a.slab.copy_(plain)
    # the same tokens, one at a time
    at = [21, 60]
    tol = 1e-5 if cache == "f32" else 2.0 ** -6
    for i in range(max(map(len, taken))):
        live = [s for s in range(2) if i < len(taken[s])]
        a.trees.set([at[s] for s in live], [1] * len(live), [a.tables[s] for s in live])
        ids = torch.tensor([taken[s][i] for s in live], device="cuda")
        for layer in range(2):
            q, k, v = (table[x][ids].view(len(live), -1, D) for x in "qkv")
            q = a.trees.append(layer, q, k, v, rope=rope, q_norm=gain, k_norm=gain)
            o = a.trees.attend(layer, q)
            for j, s in enumerate(live):
                # both are within the bounds that test_attention_is_the_formula holds them to
                assert float((o[j].float() - outs[s][i][layer].float()).abs().max()) <= tol * max(1.0, float(o[j].abs().max()))
        for s in live:
            at[s] += 1
    for s in range(2):
        for slot in range(at[s]):
            b, r = a.where(s, slot)
            assert torch.equal(got[:, b, :, :, r], a.slab[:, b, :, :, r])
    assert at == ctx
    a.close()


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
def test_one_node_over_a_decoders_cache_is_dec_attend(mode):
    from .helpers import make_pair
    from .test_gpu_attend import fill_cache, run_attend

    import numpy as np

    m, _, _ = make_pair("small", mode, max_positions=1024, max_tokens=64, max_seqs=8, n_blocks=300)
    H, D = m.shape["n_heads"], m.shape["head_dim"]
    ctxs = [1, 17, 300]
    tables = [m.blocks_for(n) for n in ctxs]
    fill_cache(m, tables, ctxs, 3, np.random.default_rng(1))
    q = torch.randn(3, H, D, device="cuda")
    want = torch.empty((3, H * D), dtype=torch.float32 if mode == "fp32" else torch.bfloat16, device="cuda")
    run_attend(m, 3, q, ctxs, tables, want)
    t = DraftTrees(m, 4, 16, 40)
    t.set([n - 1 for n in ctxs], [1, 1, 1], tables)
    got = t.attend(3, q)
    tol = 1e-5 if mode == "fp32" else 1e-2  # as test_gpu_attend
    assert float((got.float() - want.float()).abs().max()) <= tol * max(1.0, float(want.abs().max()))
    assert t.status() == 0
    t.close()
    m.close()


# ---- graphs, streams, plans ------------------------------------------------------------------------------------------


def test_captured_calls_follow_the_plan():
    w = Setup("16:8x128", "f16", [40, 200], [9, 14], seed=3)
    rope = RopeTable(128, 400)
    q, k, v = w.rand(w.N, w.H, w.D), w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    qr, out = torch.empty_like(q), torch.empty((w.N, w.H * w.D), dtype=torch.bfloat16, device="cuda")
    draft, target = torch.zeros(w.N, dtype=torch.int32, device="cuda"), torch.ones(w.N, dtype=torch.int32, device="cuda")
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (2, w.N, 2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def calls():
        w.trees.append(1, q, k, v, rope=rope, out=qr)
        w.trees.attend(1, qr, out=out)
        w.trees.commit(draft, target, out=outs)

    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
        with pytest.raises(dec.DecError) as e:  # host data cannot be captured
            w.trees.set(w.ctx, w.parents, w.tables)
        assert e.value.code == dec.DEC_EINVAL
    pool_ids = [b for t in w.tables for b in t]
    for ctx, parents in (([40, 200], [9, 14]), ([150, 31], [random_tree(9, 1), [-1] + [0] * 12 + [PAD]]), ([0, 16], [[-1] * 9, 14])):
        w.ctx, w.parents = ctx, [list(range(-1, p - 1)) if isinstance(p, int) else p for p in parents]
        ids = list(pool_ids)
        random.Random(ctx[0]).shuffle(ids)
        n0 = (ctx[0] + 9 + 15) // 16
        w.tables = [ids[:n0], ids[n0:]] if n0 + (ctx[1] + 29) // 16 <= len(ids) else w.tables
        w.trees.set(w.ctx, w.parents, w.tables)
        q.normal_()
        k.normal_()
        graph.replay()
        torch.cuda.synchronize()
        pos = torch.tensor([p or 0 for *_, p in w.nodes()], device="cuda")
        live = torch.tensor([p is not None for *_, p in w.nodes()], device="cuda")
        ref = formed(q, None, pos, 128, dec.DEC_ROPE_HALF, frequencies(128, 1e6, 0, 1, 1, 1, 1), 1.0)
        assert float((qr.double() - ref)[live].abs().max()) <= 16 * 2.0 ** -24 * float(q.abs().max())
        check(w, out, 1, qr)
        assert outs[0].tolist() == [1 if t[0] == -1 else 0 for t in w.parents]
    assert w.trees.status() == 0
    # a plan of another shape: nothing is touched, and the status says so
    w.trees.set([10], [5], [w.tables[1]])
    keep = (qr.clone(), out.clone(), w.slab.clone(), outs[1].clone())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(keep, (qr, out, w.slab, outs[1])))
    assert w.trees.status() == dec.DEC_DEV_SHAPE
    w.close()


@pytest.mark.parametrize("seqs, nodes", [(30, 7), (30, 50), (10, 200)])
def test_a_captured_call_over_plans_divided_in_other_ways(seqs, nodes):
    """The same nodes over contexts whose units stay whole, are joined in place, or go through the merge kernel."""
    trees = [random_tree(nodes, i) for i in range(seqs)]
    w = Setup("16:8x128", "f16", [1700 + i for i in range(seqs)], trees, seed=5)
    q = w.rand(w.N, w.H, w.D)
    tables, out = w.tables, torch.empty((w.N, w.H * w.D), dtype=torch.float16, device="cuda")
    plans = [[1700 + i for i in range(seqs)], [10 + i for i in range(seqs)], [900] * seqs, [0] * (seqs - 1) + [1700 + seqs - 1]]
    for first in (0, 1):
        w.ctx = plans[first]
        w.trees.set(w.ctx, w.parents, tables)
        w.trees.attend(0, q, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.trees.attend(0, q, out=out)
        for w.ctx in plans + plans[::-1]:
            w.trees.set(w.ctx, w.parents, tables)
            out.fill_(float("nan"))
            graph.replay()
            graph.replay()
            got = out.clone()
            w.trees.attend(0, q, out=out)
            # the same parts, but a merge kernel that was chosen at the capture may add them in another order: fp32 sums of up
            # to 64 parts of values of about 1 (64 half steps), and then up to one step of the output apart
            off = (got.float() - out.float()).abs()
            assert bool((off <= 2 * 2.0 ** -11 * out.float().abs() + 64 * 2.0 ** -24).all())
        for w.ctx in plans:
            w.trees.set(w.ctx, w.parents, tables)
            graph.replay()
            check(w, out, 0, q, sorted(random.Random(4).sample(range(w.N), 20)))
        del graph
    w.close()


def test_a_replay_that_outgrows_its_rotary_table_says_so():
    w = Setup("8:4x64", "f16", [10], [4], seed=3, extra_blocks=0)
    rope = RopeTable(64, 14)
    q = w.rand(4, w.H, w.D)
    w2 = Setup("8:4x64", "f16", [30], [4], seed=3)
    out = torch.empty_like(q)
    w2.trees.set([10], [4], w2.tables)
    w2.trees.append(0, q, None, None, rope=rope, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w2.trees.append(0, q, None, None, rope=rope, out=out)
    w2.trees.set([30], [4], w2.tables)
    with pytest.raises(dec.DecError):  # a direct call is refused
        w2.trees.append(0, q, None, None, rope=rope, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert w2.trees.status() == dec.DEC_DEV_BOUNDS
    w2.close()
    w.close()


def test_two_plans_on_two_streams():
    a = Setup("16:8x128", "f16", [900, 700], [random_tree(30, 1), 20], seed=1)
    b = Setup("16:8x128", "f16", [1500], [random_tree(64, 2)], seed=2)
    qa, qb = a.rand(a.N, a.H, a.D), b.rand(b.N, b.H, b.D)
    want = a.trees.attend(0, qa).clone(), b.trees.attend(0, qb).clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        ga, gb = a.trees.attend(0, qa, stream=sa), b.trees.attend(0, qb, stream=sb)
        sa.synchronize()
        sb.synchronize()
        assert torch.equal(ga, want[0]) and torch.equal(gb, want[1])
    a.close()
    b.close()


@pytest.mark.parametrize("nodes", [6, 50])
def test_full_batches_on_two_streams(nodes):
    """Batches whose units are joined by the CTAs that start them, side by side on one GPU."""
    a, b = (Setup("16:8x128", "f16", [900 + 7 * i for i in range(30)], [nodes] * 30, seed=k) for k in (1, 2))
    qa, qb = a.rand(a.N, a.H, a.D), b.rand(b.N, b.H, b.D)
    want = a.trees.attend(0, qa).clone(), b.trees.attend(0, qb).clone()
    check(a, want[0], 0, qa, sorted(random.Random(1).sample(range(a.N), 20)))
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        got = [(a.trees.attend(0, qa, stream=sa), b.trees.attend(0, qb, stream=sb)) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)
    a.close()
    b.close()


@pytest.mark.parametrize("shape", ["16:8x128", "8:2x128", "8:4x64", "4:2x32"])
def test_trees_of_every_width_in_one_batch(shape):
    """Sequences of one to eight row tiles share the CTAs; some contexts are a few keys, some fill many tiles."""
    counts = [256, 1, 70, 129, 33, 17, 200, 0, 65, 3]
    ctx = [0, 2000, 500, 7, 130, 64, 1000, 9, 3, 300]
    w = Setup(shape, "f16", ctx, [random_tree(n, n) if n else 0 for n in counts], seed=6)
    q = w.rand(w.N, w.H, w.D)
    out = w.trees.attend(1, q)
    check(w, out, 1, q, sorted(random.Random(2).sample(range(w.N), 120)))
    w.close()


def test_the_same_inputs_give_the_same_bits():
    w = Setup("16:8x128", "f16", [1234, 77], [random_tree(64, 1), 3], seed=1)
    q = w.rand(w.N, w.H, w.D)
    first = w.trees.attend(1, q).clone()
    for _ in range(10):
        assert torch.equal(w.trees.attend(1, q), first)
    w.close()


# ---- refusals ---------------------------------------------------------------------------------------------------------


def test_refusals():
    w = Setup("8:4x64", "f16", [20], [6], seed=1)
    L, t, N = w.trees.L, w.trees, w.N
    q = w.rand(N, w.H, w.D)
    out = torch.zeros((N, w.H * w.D), dtype=torch.bfloat16, device="cuda")
    P, O = q.data_ptr(), out.data_ptr()
    ld = w.H * w.D

    def attend(layer=0, q=P, qt=0, ldq=ld, out=O, ot=2, ldo=ld):
        return L.dec_tree_attend(t.handle, layer, q, qt, ldq, out, ot, ldo, None)

    assert attend() == dec.DEC_OK
    for bad in ({"layer": -1}, {"layer": 2}, {"q": None}, {"out": None}, {"qt": 3}, {"qt": -1}, {"ot": 5}, {"ot": 0}, {"ldq": ld - 4}, {"ldq": ld + 2},
                {"ldo": 0}, {"ldo": ld + 1}, {"q": P + 4}, {"out": O + 4}, {"q": O, "qt": 2}):
        assert attend(**bad) == dec.DEC_EINVAL, bad
        assert L.dec_last_error()
    rope = RopeTable(64, 26)
    short = RopeTable(64, 25)
    k = w.rand(N, w.Hkv, w.D)
    assert w.trees.append(0, q, k, k, rope=rope).shape == q.shape
    with pytest.raises(dec.DecError) as e:
        w.trees.append(0, q, k, k, rope=short)
    assert e.value.code == dec.DEC_ERANGE
    with pytest.raises(dec.DecError):
        w.trees.append(0, q, k, k, rope=RopeTable(128, 26))  # more channels than the head has
    for call in (lambda: w.trees.append(0, None, None, None), lambda: w.trees.append(0, None, k, None), lambda: w.trees.append(2, q, k, k)):
        with pytest.raises(dec.DecError) as e:
            call()
        assert e.value.code == dec.DEC_EINVAL
    for call in (lambda: w.trees.attend(0, q[:3]), lambda: w.trees.attend(0, q.double()), lambda: w.trees.attend(0, q.cpu()), lambda: w.trees.attend(0, q.transpose(1, 2)),
                 lambda: w.trees.append(0, q, k.half(), k), lambda: w.trees.append(0, q, k, k, q_norm=torch.ones(3, device="cuda")),
                 lambda: w.trees.commit(torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    ids = torch.zeros(N, dtype=torch.int32, device="cuda")
    assert L.dec_tree_commit(t.handle, None, ids.data_ptr(), None, ids.data_ptr(), ids.data_ptr(), ids.data_ptr(), None) == dec.DEC_EINVAL
    # a refused batch leaves the plan as it was
    want = w.trees.attend(0, q).clone()
    for ctx, parents, tables in (([20, 20], [3, 3], [w.tables[0]] * 2), ([20], [7], w.tables), ([5], [[-1, 1]], w.tables), ([70], [1], [w.tables[0] * 4])):
        with pytest.raises(dec.DecError):
            w.trees.set(ctx, parents, tables)
    assert torch.equal(w.trees.attend(0, q), want)
    h = C.c_void_p()
    for args in ((0, 5, 5), (1, 0, 5), (1, 5, 0), (1, 1 << 21, 5)):
        assert L.dec_tree_create(w.pool.pool, *args, C.c_void_p(1 << 40), 1 << 40, C.byref(h)) != dec.DEC_OK
    assert L.dec_tree_create(w.pool.pool, 1, 5, 5, C.c_void_p(256), 100, C.byref(h)) == dec.DEC_EINVAL
    assert L.dec_tree_create(w.pool.pool, 1, 5, 5, C.c_void_p(100), 1 << 40, C.byref(h)) == dec.DEC_EINVAL
    fresh = DraftTrees(w.pool, 1, 6, 4)
    assert L.dec_tree_attend(fresh.handle, 0, P, 0, ld, O, 2, ld, None) == dec.DEC_EINVAL  # no trees yet
    fresh.close()
    w.close()
