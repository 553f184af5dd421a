"""Draft trees over a cache held in 8 bits on the GPU: attention, the append
that quantises, the commit between pages of other scales and the reading back,
against plain implementations in 64 bits, and the calls that could go wrong:
scales far apart, memory that no call has written, pages that end anywhere,
padding, values that are not finite, captured and replayed calls, streams."""

import ctypes as C
import math
import random

import pytest

torch = pytest.importorskip("torch")

from decoder_qwen3_step_gb300 import dec  # noqa: E402
from decoder_qwen3_step_gb300.trees import DraftTrees, KvPool, RopeTable  # noqa: E402
from tests.q8_reference import E_MIN, KINDS, codes_of, log2, need, numbers, rounded, two  # noqa: E402
from tests.test_gpu_trees import BATCHES, HALF_STEP, PAD, SHAPES, formed, frequencies, random_tree, walk  # noqa: E402

pytestmark = pytest.mark.gpu


class Setup8:
    """A pool of random 8-bit pages in random order, and a plan of the given trees."""

    def __init__(self, shape, kind, ctx, parents, layers=2, seed=0, spare=3, extra_blocks=0, spread=1, max_tokens=None):
        self.H, self.Hkv, self.D = SHAPES[shape]
        self.kind, self.layers = kind, layers
        rng = random.Random(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.ctx, self.parents = list(ctx), [list(range(-1, p - 1)) if isinstance(p, int) else list(p) for p in parents]
        need_blocks = [(c + len(p) + 15) // 16 for c, p in zip(self.ctx, self.parents)]
        self.blocks = sum(need_blocks) + spare + extra_blocks
        self.shape = {"vocab": 512, "d_model": 64, "n_layers": layers, "n_heads": self.H, "n_kv_heads": self.Hkv, "head_dim": self.D, "ff_hidden": 64}
        n = layers * self.blocks * 2 * self.Hkv * 16 * self.D
        at = (n + 255) // 256 * 256
        self.buf = torch.zeros(at + layers * self.blocks * self.Hkv * 2 * 4, dtype=torch.uint8, device="cuda")
        self.codes = self.buf[:n].view(layers, self.blocks, 2, self.Hkv, 16, self.D)
        self.scales = self.buf[at:].view(torch.float32).view(layers, self.blocks, self.Hkv, 2)
        for layer in range(layers):
            x = torch.randn((self.blocks, 2, self.Hkv, 16, self.D), generator=self.g).double().cuda()
            x *= two(torch.randint(-spread, spread + 1, (self.blocks, 2, self.Hkv, 1, 1), generator=self.g).cuda())
            e = need(x.abs().amax((-2, -1)), kind)
            self.codes[layer] = codes_of(x, e[..., None, None], kind)
            self.scales[layer] = two(e).transpose(1, 2).float()
        self.pool = KvPool(self.shape, dec.DEC_BF16_F16KV, self.blocks, max_positions=40960, slabs=self.buf, kv_type=KINDS[kind])
        ids = self.pool.alloc(self.blocks)
        rng.shuffle(ids)
        self.tables = [[ids.pop() for _ in range(n)] for n in need_blocks]
        self.N = sum(len(p) for p in self.parents)
        self.trees = DraftTrees(self.pool, max(len(self.ctx), 1), max_tokens or self.N, max(need_blocks + [1]) + 2)
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

    def values(self):
        """What the codes stand for, in 64 bits: [layers, blocks, 2, KV heads, 16, D]."""
        return numbers(self.codes, self.kind) * self.scales.double().transpose(2, 3)[..., None, None]

    def rows(self, layer, s, slots):
        """K and V [slots, KV heads, D] and their scales [slots, KV heads]."""
        b = torch.tensor([self.where(s, x)[0] for x in slots], dtype=torch.long, device="cuda")
        r = torch.tensor([x % 16 for x in slots], dtype=torch.long, device="cuda")
        c, sc = numbers(self.codes[layer][b, :, :, r], self.kind), self.scales[layer][b].double()
        return c[:, 0] * sc[:, :, :1], c[:, 1] * sc[:, :, 1:], sc[:, :, 0], sc[:, :, 1]

    def close(self, status=0):
        torch.cuda.synchronize()
        assert self.trees.status() == status
        self.trees.close()
        self.pool.close()


def check(w, out, layer, q, only=None):
    """Against the formula in 64 bits, node by node, within what the roundings allow."""
    G = w.H // w.Hkv
    got_all = out.view(w.N, w.H, w.D).double()
    off2 = ref2 = 0.0
    for n, s, i, slot, pos in w.nodes():
        if pos is None or (only is not None and n not in only):
            continue
        k, v, _, vs = (x.repeat_interleave(G, 1) for x in w.rows(layer, s, w.seen(s, i)))
        qn = q[n].double()
        sc = torch.einsum("hd,khd->hk", qn, k) / math.sqrt(w.D)
        size = torch.einsum("hd,khd->hk", qn.abs(), k.abs()) / math.sqrt(w.D)  # what the score's roundings are relative to
        p = torch.softmax(sc, -1)
        ref = torch.einsum("hk,khd->hd", p, v)
        spread = torch.einsum("hk,khd->hd", p, v.abs()).amax(-1, keepdim=True)
        # a score off by e changes its weight by a factor within exp(+-e), the sum likewise; fp32: products and partial sums,
        # D + 4 half steps of their size, the exponential's argument and result 4 more; f16 queries and weights: half a step
        # each; a sum over the keys rounds like sqrt(keys) half steps or less, 64 cover it
        worst = (p * size).sum(-1, keepdim=True) + size.amax(-1, keepdim=True)
        tol = ((w.D + 8) * 2.0 ** -24 * worst + (64 + 8) * 2.0 ** -24 + 2.0 ** -11 * worst + 2 * 2.0 ** -11) * spread * 1.01 + 1e-300
        # weights times a page's scale that are subnormal in f16: half of their step, 2^-25 of a reference that is at most
        # the largest of them, times the codes
        tol = tol + 2.0 ** -25 * ((p * vs.T).amax(-1)[:, None] * (v.abs() / vs[:, :, None]).sum(0)).amax(-1, keepdim=True)
        got = got_all[n]
        off = (got - ref).abs()
        allowed = tol + HALF_STEP[out.dtype] * (ref.abs() + tol)
        assert bool(torch.isfinite(got).all())
        assert bool((off <= allowed).all()), (n, s, i, float((off / allowed).max()))
        off2, ref2 = off2 + float((off / spread).square().sum()), ref2 + float((ref / spread).square().sum())
    # and as a whole the roundings do not pull one way: two half steps of bf16's cover them
    assert math.sqrt(off2) <= 2 * 2.0 ** -8 * math.sqrt(ref2) + 1e-12


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_attention_is_the_formula(batch, shape, kind):
    ctx, parents = BATCHES[batch]
    w = Setup8(shape, kind, ctx, parents, seed=len(batch))
    q = w.rand(w.N, w.H, w.D)
    out = torch.full((w.N, w.H * w.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    w.trees.attend(1, q, out=out)
    check(w, out, 1, q, set(random.Random(1).sample(range(w.N), min(w.N, 40))))
    pads = [n for n, _, _, _, pos in w.nodes() if pos is None]
    assert not bool(out[pads].any())
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape, nodes", [("16:8x128", 3), ("16:8x128", 40), ("16:8x128", 200), ("8:4x64", 90), ("4:2x32", 20)])
def test_pages_whose_scales_lie_far_apart(shape, nodes, kind):
    ctx, parents = [260, 1000], [random_tree(nodes, 1), random_tree(max(nodes // 2, 1), 2)]
    w = Setup8(shape, kind, ctx, parents, seed=4)
    # values of 2^-38 .. 2^34 beside each other, pages of zeros, keys of all sizes that leave the scores alone
    e = torch.randint(-38, 28, w.scales[..., 1].shape, generator=w.g).cuda()
    w.scales[..., 1] = two(e)
    zero = torch.rand(w.scales[..., 1].shape, generator=w.g).cuda() < 0.1
    w.codes[:, :, 1][zero] = 0
    w.scales[..., 1][zero] = 2.0 ** E_MIN
    q = w.rand(w.N, w.H, w.D)
    check(w, w.trees.attend(0, q), 0, q, set(range(0, w.N, max(w.N // 20, 1))))
    small = two(torch.randint(-6, 1, w.scales[..., 0].shape, generator=w.g).cuda()).float()
    w.scales[..., 0] *= small
    check(w, w.trees.attend(1, q), 1, q, set(range(0, w.N, max(w.N // 20, 1))))
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape, nodes", [("8:4x64", 23), ("16:8x128", 4), ("16:8x128", 23), ("16:8x128", 150), ("4:2x32", 23)])
def test_memory_that_no_call_has_written_changes_nothing(shape, nodes, kind):
    ctx, parents = [37, 70, 0, 5], [random_tree(nodes, 1), [-1, 0, 0, 1, PAD, PAD], random_tree(nodes + 7, 2), [PAD] * 30]
    w = Setup8(shape, kind, ctx, parents, seed=9)
    q = w.rand(w.N, w.H, w.D)
    clean = w.trees.attend(0, q).clone()
    # everything that belongs to no token: the rest of the last pages, padding's slots, the other pages, the other layer
    mask = torch.ones(w.codes.shape[1], 16, dtype=torch.bool, device="cuda")
    for s in range(len(ctx)):
        for slot in range(w.ctx[s] + len(w.parents[s])):
            if slot < w.ctx[s] or w.parents[s][slot - w.ctx[s]] != PAD:
                b, r = w.where(s, slot)
                mask[b, r] = False
    for code in (0x7F, 0xFF, 0x80):  # no number in e4m3
        w.codes[0].permute(0, 3, 1, 2, 4)[mask] = code
        w.codes[1] = code
        for scale in (float("nan"), float("inf"), -1.0, 0.0):
            w.scales[0][mask.all(1)] = scale
            w.scales[1] = scale
            assert torch.equal(w.trees.attend(0, q), clean), (code, scale)
    # queries that are NaN give NaN, and leave the others alone
    bad = q.clone()
    bad[2, 0, 3] = float("nan")
    got = w.trees.attend(0, bad).view(w.N, w.H, w.D)
    assert bool(torch.isnan(got[2, 0]).all())
    got[2, 0] = clean.view(w.N, w.H, w.D)[2, 0]
    assert torch.equal(got.view_as(clean), clean)
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape, nodes", [("16:8x128", 3), ("16:8x128", 40), ("16:8x128", 200), ("8:4x64", 40), ("8:2x128", 2), ("4:2x32", 20)])
@pytest.mark.parametrize("spread", [4.0, 40.0, 1000.0])
def test_scores_far_apart(spread, shape, nodes, kind):
    """Scores that rise along the keys by tens to tens of thousands: a row's reference is raised again and again, within the
    tiles, too, and one key takes nearly all the weight."""
    ctx, parents = [700, 129], [random_tree(nodes, 1), nodes]
    w = Setup8(shape, kind, ctx, parents, seed=11)
    # the keys' first channel grows with the position, up or down by head; queries are large there
    for s in range(2):
        for slot in range(0, w.ctx[s] + len(w.parents[s])):
            b, r = w.where(s, slot)
            ramp = (slot % 128) / 128 if slot % 3 else 0.5
            codes = codes_of(torch.full((w.Hkv,), ramp * 100, dtype=torch.float64), torch.zeros(w.Hkv, dtype=torch.float64), kind)
            w.codes[0, b, 0, :, r, 0] = torch.where(torch.arange(w.Hkv) % 2 == 0, codes, codes_of(torch.full((w.Hkv,), 100 - ramp * 100, dtype=torch.float64), torch.zeros(w.Hkv, dtype=torch.float64), kind)).cuda()
    q = w.rand(w.N, w.H, w.D)
    q[..., 0] = spread * (1 + torch.rand(q[..., 0].shape, generator=w.g).cuda())
    check(w, w.trees.attend(0, q), 0, q, set(range(0, w.N, max(w.N // 20, 1))))
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("scale", [1e30, 1e-30, 70000.0, 0.0])
def test_queries_of_any_magnitude(scale, kind):
    for nodes in (3, 60):
        w = Setup8("16:8x128", kind, [100, 19], [nodes, nodes], seed=2)
        q = w.rand(w.N, w.H, w.D) * scale
        out = w.trees.attend(0, q).view(w.N, w.H, w.D).double()
        assert bool(torch.isfinite(out).all())
        if scale == 0.0 or scale == 1e-30:  # all weights alike
            for n, s, i, _, _ in w.nodes():
                v = w.rows(0, s, w.seen(s, i))[1].repeat_interleave(2, 1)
                ref, spread = v.mean(0), v.abs().mean(0).amax(-1, keepdim=True)
                assert bool(((out[n] - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 80 * 2.0 ** -24) * spread).all())
        w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("in_type", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nodes", [5, 40, 150])
def test_types_strides_and_rows_behind_the_last(in_type, nodes, kind):
    w = Setup8("16:8x128", kind, [90, 3], [nodes, nodes - 3], seed=7)
    wide = torch.randn((w.N + 2, w.H * w.D + 24), generator=w.g).cuda().to(in_type)
    q = wide[:w.N, 8:8 + w.H * w.D]
    for out_type in (torch.bfloat16, torch.float16):
        big = torch.full((w.N + 2, w.H * w.D + 12), 7.0, dtype=out_type, device="cuda")
        out = big[:w.N, 4:4 + w.H * w.D]
        w.trees.attend(0, q, out=out)
        check(w, out.contiguous(), 0, q.reshape(w.N, w.H, w.D), set(range(0, w.N, max(w.N // 20, 1))))
        assert bool((big[w.N:] == 7).all() and (big[:, :4] == 7).all() and (big[:, 4 + w.H * w.D:] == 7).all())
    with pytest.raises(dec.DecError):
        w.trees.attend(0, q, out_type=torch.float32)
    w.close()


# ---- append ---------------------------------------------------------------------------------------------------


def expected_pages(w, layer, kv):
    """Codes and exponents of `layer` after an append of kv [nodes, 2, KV heads, D] (64 bits), from what is there now."""
    codes, e = w.codes[layer].clone(), log2(w.scales[layer]).transpose(1, 2).clone()  # [blocks, 2, KV heads]
    pages = {}
    for n, s, i, slot, pos in w.nodes():
        pages.setdefault((s, slot // 16), []).append((n, slot % 16, pos))
    for (s, p), rows in pages.items():
        b = w.tables[s][p]
        rows = [(n, r) for n, r, pos in rows if pos is not None]
        cached = max(0, min(16, w.ctx[s] - p * 16))
        top = torch.zeros((2, w.Hkv), dtype=torch.float64, device="cuda")
        for n, _ in rows:
            top = torch.maximum(top, torch.where(torch.isfinite(kv[n]), kv[n].abs(), 0.0).amax(-1))
        new = need(top, w.kind)
        if cached:
            new = torch.maximum(new, e[b])
            again = codes_of(numbers(codes[b, :, :, :cached], w.kind) * two(e[b])[..., None, None], new[..., None, None], w.kind)
            codes[b, :, :, :cached] = torch.where((new > e[b])[..., None, None], again, codes[b, :, :, :cached])
        e[b] = new
        for n, r in rows:
            codes[b, :, :, r] = codes_of(torch.nan_to_num(kv[n], nan=0.0, posinf=1e300, neginf=-1e300), new[..., None], w.kind)
    return codes, e


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_append_without_rotation_gives_the_nearest_codes(batch, shape, kind):
    ctx, parents = BATCHES[batch]
    w = Setup8(shape, kind, ctx, parents, seed=len(batch) + 1)
    # magnitudes that raise some pages' scales and not others', ties between codes, both ends of the range
    k, v = w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    k *= torch.exp2(torch.randint(-3, 4, (w.N, w.Hkv, 1), generator=w.g).float()).cuda()
    v[::3] = (v[::3] * 32).round() / 64
    want = expected_pages(w, 1, torch.stack([k, v], 1).double())
    other = w.codes[0].clone(), w.scales[0].clone()
    w.trees.append(1, None, k, v)
    assert torch.equal(log2(w.scales[1]).transpose(1, 2), want[1])
    assert torch.equal(w.codes[1], want[0])
    assert torch.equal(w.codes[0], other[0]) and torch.equal(w.scales[0], other[1])
    w.trees.append(1, None, k, v)  # the same again: nothing changes
    assert torch.equal(w.codes[1], want[0])
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", ["4:2x32", "12:3x32", "8:4x64", "16:8x128"])
def test_append_with_padding_in_pages_of_any_number_of_rows(shape, kind):
    """Pages of 1 .. 16 rows, at a page's start and at its end, padding first, everywhere but last, and anywhere."""
    ctx, parents = [], []
    rng = random.Random(7)
    for n in range(1, 17):
        for pads in ({0}, set(range(n - 1)), {i for i in range(n) if rng.random() < 0.5}):
            for c in (32, 48 - n):
                ctx.append(c)
                parents.append([PAD if i in pads else -1 for i in range(n)])
    w = Setup8(shape, kind, ctx, parents, seed=4)
    k, v = w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    k *= torch.exp2(torch.randint(-3, 4, (w.N, w.Hkv, 1), generator=w.g).float()).cuda()
    want = expected_pages(w, 0, torch.stack([k, v], 1).double())
    w.trees.append(0, None, k, v)
    assert torch.equal(log2(w.scales[0]).transpose(1, 2), want[1])
    assert torch.equal(w.codes[0], want[0])
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("in_type", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape, rot, layout", [("4:2x32", 8, dec.DEC_ROPE_HALF), ("16:8x128", 128, dec.DEC_ROPE_HALF), ("16:8x128", 72, dec.DEC_ROPE_INTERLEAVED), ("8:4x64", 48, dec.DEC_ROPE_HALF),
                                                ("5:5x64", 64, dec.DEC_ROPE_INTERLEAVED), ("8:2x128", 128, dec.DEC_ROPE_HALF)])
def test_append_is_the_formula(shape, rot, layout, in_type, kind):
    w = Setup8(shape, kind, [37, 0, 250, 15], [random_tree(40, 1), 3, [-1, PAD, 0, 0, PAD], 1], seed=rot)
    H, Hkv, D = w.H, w.Hkv, w.D
    raw = torch.randn((w.N, (H + 2 * Hkv) * D + 8), generator=w.g).cuda().to(in_type)
    q, k, v = raw[:, :H * D], raw[:, H * D:(H + Hkv) * D], raw[:, (H + Hkv) * D:(H + 2 * Hkv) * D]
    gq, gk = 1 + 0.1 * w.rand(D), 1 + 0.1 * w.rand(D)
    rope = RopeTable(rot, 400, layout=layout, scaling=dec.DEC_ROPE_LINEAR, factor=4.0)
    freq = frequencies(rot, 1e6, dec.DEC_ROPE_LINEAR, 4.0, 0, 0, 0)
    pos = torch.tensor([p or 0 for *_, p in w.nodes()], device="cuda")
    pads = torch.tensor([p is None for _, _, _, _, p in w.nodes()], device="cuda")
    fq = formed(q.reshape(w.N, H, D), gq, pos, rot, layout, freq, 1.0)
    fk = formed(k.reshape(w.N, Hkv, D), gk, pos, rot, layout, freq, 1.0)
    before = w.codes.clone()
    codes, e = expected_pages(w, 0, torch.stack([fk, v.reshape(w.N, Hkv, D).double()], 1))
    got_q = w.trees.append(0, q, k, v, rope=rope, q_norm=gq, k_norm=gk, q_type=torch.float32)
    # the table's rounding, two products and their sum, with a norm the D squares' sum and five operations more
    eps = (4 + D / 2 + 6) * 2.0 ** -24
    size = fq.abs() + 2 * formed(q.reshape(w.N, H, D), gq, pos, 0, 0, freq, 1.0).abs().amax(-1, keepdim=True)
    assert bool(((got_q.double() - fq).abs() <= eps * size + HALF_STEP[torch.float32] * fq.abs())[~pads].all())
    assert not bool(got_q[pads].any())
    got_e = log2(w.scales[0]).transpose(1, 2)
    # an exponent may differ where the largest magnitude lies within fp32's rounding of a border: not with these inputs
    assert torch.equal(got_e, e)
    step = two(e)[..., None, None] * (1.0 if kind == "i8" else 32.0)  # of the largest codes
    a, b = numbers(w.codes[0], kind) * two(e)[..., None, None], numbers(codes, kind) * two(e)[..., None, None]
    assert bool(((a - b).abs() <= step).all())  # the neighbouring code where the value is next to a tie
    # its share: a value is within eps of a tie, of a step that is 2^-7 (i8) or 2^-4 (e4m3, of the value) or more
    assert int((w.codes[0] != codes).sum()) <= 4 + 8 * eps * 2.0 ** 7 * codes.numel()
    assert torch.equal(w.codes[0, :, 1], codes[:, 1])  # values are not rotated
    assert torch.equal(w.codes[1], before[1])
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("in_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape, rot, layout", [("4:2x32", 32, dec.DEC_ROPE_INTERLEAVED), ("4:2x32", 8, dec.DEC_ROPE_HALF), ("16:8x128", 128, dec.DEC_ROPE_HALF), ("16:8x128", 72, dec.DEC_ROPE_INTERLEAVED),
                                                ("8:4x64", 48, dec.DEC_ROPE_HALF), ("8:2x128", 128, dec.DEC_ROPE_HALF)])
def test_every_appended_code_lies_between_the_roundings(shape, rot, layout, in_type, kind):
    """A key's code is one that a value within fp32's reach of the formula rounds to, nothing else is written."""
    w = Setup8(shape, kind, [37, 0, 250, 15], [random_tree(40, 1), 3, [-1, PAD, 0, 0, PAD], 1], seed=rot, spread=0)
    Hkv, D = w.Hkv, w.D
    k, v = (torch.randn((w.N, Hkv, D), generator=w.g).cuda().to(in_type) for _ in range(2))
    g = 1 + 0.1 * w.rand(D)
    rope = RopeTable(rot, 400, layout=layout, scaling=dec.DEC_ROPE_LINEAR, factor=4.0)
    freq = frequencies(rot, 1e6, dec.DEC_ROPE_LINEAR, 4.0, 0, 0, 0)
    pos = torch.tensor([p or 0 for *_, p in w.nodes()], device="cuda")
    fk = formed(k, g, pos, rot, layout, freq, 1.0)
    # as in test_append_is_the_formula: the table's rounding, two products and their sum, the norm
    eps = (4 + D / 2 + 6) * 2.0 ** -24
    off = eps * (fk.abs() + 2 * formed(k, g, pos, 0, 0, freq, 1.0).abs().amax(-1, keepdim=True))
    off = torch.stack([off, torch.zeros_like(off)], 1)  # values are rounded to codes only
    kv = torch.stack([fk, v.double()], 1)
    codes, was = w.codes[0].clone(), log2(w.scales[0]).transpose(1, 2).clone()  # [blocks, 2, KV heads]
    w.trees.append(0, None, k, v, rope=rope, k_norm=g)
    got, e = numbers(w.codes[0], kind), log2(w.scales[0]).transpose(1, 2)
    untouched = torch.ones_like(codes, dtype=torch.bool)
    pages = {}
    for n, s, i, slot, p in w.nodes():
        pages.setdefault((s, slot // 16), []).append((n, slot % 16, p))
    for (s, p), rows in pages.items():
        b, live = w.tables[s][p], [(n, r) for n, r, at in rows if at is not None]
        cached = max(0, min(16, w.ctx[s] - p * 16))
        least = was[b] if cached else torch.full_like(was[b], E_MIN)
        at = torch.tensor([n for n, _ in live], dtype=torch.long, device="cuda")
        for bound, side in ((kv[at].abs() - off[at], 1), (kv[at].abs() + off[at], -1)):
            edge = torch.maximum(least, need(bound.clamp(min=0).amax((0, -1)), kind)) if live else least
            assert bool((side * (e[b] - edge) >= 0).all())
        if cached:
            again = codes_of(numbers(codes[b, :, :, :cached], kind) * two(was[b])[..., None, None], e[b][..., None, None], kind)
            rose = (e[b] > was[b])[..., None, None]
            assert torch.equal(w.codes[0][b, :, :, :cached], torch.where(rose, again, codes[b, :, :, :cached]))
            untouched[b, :, :, :cached] = False
        for n, r in live:
            scale = two(e[b])[..., None]
            low, high = (rounded((kv[n] + side * off[n]) / scale, kind) for side in (-1, 1))
            mine = got[b, :, :, r]
            assert bool(((low <= mine) & (mine <= high)).all()), (n, r)
            untouched[b, :, :, r] = False
    assert torch.equal(w.codes[0][untouched], codes[untouched])
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape, nodes", [("16:8x128", 3), ("8:4x64", 40), ("4:2x32", 256), ("12:3x32", 20)])
def test_queries_in_place_and_parts_alone(shape, nodes, kind):
    w = Setup8(shape, kind, [37, 5], [nodes, max(nodes // 3, 1)], seed=3)
    rope = RopeTable(w.D, 400)
    q, k, v = w.rand(w.N, w.H, w.D), w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    g = 1 + 0.1 * w.rand(w.D)
    start = w.buf.clone()
    both = w.trees.append(0, q, k, v, rope=rope, q_norm=g, k_norm=g)
    whole = w.buf.clone()
    w.buf.copy_(start)
    w.trees.append(0, None, k, v, rope=rope, k_norm=g)
    assert torch.equal(w.buf, whole)
    assert torch.equal(w.trees.append(0, q, None, None, rope=rope, q_norm=g), both)
    assert torch.equal(w.buf, whole)
    same = q.clone()
    w.trees.append(0, same, None, None, rope=rope, q_norm=g, out=same)
    assert torch.equal(same, both)
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("nodes", [2, 20, 100])
def test_a_page_next_to_one_with_a_far_larger_scale_keeps_its_values(nodes, kind):
    """Scales 2^28 apart within 128 slots, the large page's weights as good as zero: rows are the small pages' values."""
    w = Setup8("16:8x128", kind, [128 * 3], [nodes], seed=3)
    q = w.rand(w.N, w.H, w.D)
    q[..., 0] = 60.0
    w.codes[0, :, 0, :, :, 0] = codes_of(torch.tensor(100.0, dtype=torch.float64), torch.tensor(0.0), kind).item()  # every score up
    w.scales[0, :, :, 0] = 1.0
    for p in (1, 9, 20):  # one page of each tile: hidden by low scores, its values 2^28 times the others'
        b = w.tables[0][p]
        w.codes[0, b, 0, :, :, 0] = codes_of(torch.tensor(-100.0, dtype=torch.float64), torch.tensor(0.0), kind).item()
        w.scales[0, b, :, 1] *= 2.0 ** 28 / 2
    check(w, w.trees.attend(0, q), 0, q, set(range(0, w.N, max(w.N // 20, 1))))
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
def test_a_page_filled_token_by_token_loses_less_than_a_step(kind):
    """16 calls of one token, growing: every value ends within one step of its page's final scale, and e is that of one call."""
    w = Setup8("16:8x128", kind, [32], [1], seed=3, extra_blocks=2)
    x = w.rand(16, 2, w.Hkv, w.D) * torch.exp2(torch.arange(16, device="cuda").float() / 3 - 4)[:, None, None, None]
    for i in range(16):
        w.trees.set([32 + i], [1], w.tables)
        w.trees.append(0, None, x[i:i + 1, 0], x[i:i + 1, 1])
    block = w.tables[0][2]
    e = log2(w.scales[0, block]).T  # [2, KV heads]
    assert torch.equal(e, need(x.double().abs().amax((0, -1)), kind))
    got = numbers(w.codes[0, block], kind) * two(e)[..., None, None]  # [2, KV heads, 16, D]
    want = x.double().permute(1, 2, 0, 3)
    if kind == "i8":
        allowed = two(e)[..., None, None].expand_as(want)  # 1/2 + 1/4 + .. steps
    else:  # a code keeps its bits until it is subnormal (steps of 2^-9): half a step of the value, then as above
        allowed = 2.0 ** -4 * want.abs() + 2.0 ** -9 * two(e)[..., None, None]
    assert bool(((got - want).abs() <= allowed).all())
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("ctx", [32, 37])
def test_values_that_are_not_finite_are_cut_and_told(kind, ctx):
    w = Setup8("8:4x64", kind, [ctx], [20], seed=5)
    k, v = w.rand(20, 4, 64), w.rand(20, 4, 64)
    k[3, 1, 7], k[4, 1, 8], v[5, 2, 9], v[18, 0, 63] = float("inf"), -float("inf"), float("nan"), float("inf")
    want = expected_pages(w, 0, torch.stack([k, v], 1).double())
    w.trees.append(0, None, k, v)
    assert w.trees.status() == dec.DEC_DEV_NONFINITE
    assert torch.equal(w.codes[0], want[0]) and torch.equal(log2(w.scales[0]).transpose(1, 2), want[1])
    # magnitudes past both ends of the scales, and zeros
    k = w.rand(20, 4, 64) * 1e38
    v = torch.zeros(20, 4, 64, device="cuda")
    k[:, 0] *= 0
    k[:, 1] *= 1e-38 * 1e-30
    want = expected_pages(w, 0, torch.stack([k, v], 1).double())
    w.trees.append(0, None, k, v)
    assert torch.equal(w.codes[0], want[0]) and torch.equal(log2(w.scales[0]).transpose(1, 2), want[1])
    # a normal deviate above 3.4 times 1e38 is infinite in fp32: told again
    w.close(0 if bool(torch.isfinite(k).all()) else dec.DEC_DEV_NONFINITE)


@pytest.mark.parametrize("kind", list(KINDS))
def test_a_page_of_nothing_but_padding_has_a_scale(kind):
    w = Setup8("8:4x64", kind, [30], [[PAD] * 2 + [-1] + [PAD] * 20], seed=5)
    w.scales[:] = float("nan")
    w.scales[0, w.tables[0][1]] = 0.5
    before = w.codes.clone()
    k, v = w.rand(w.N, 4, 64), w.rand(w.N, 4, 64)
    w.trees.append(0, None, k, v)
    assert bool((w.scales[0, w.tables[0][1]] == 0.5).all())  # padding at the end of a page with cached tokens
    assert bool((w.scales[0, w.tables[0][3]] == 2.0 ** E_MIN).all())
    changed = (w.codes != before).any(-1)  # [layers, blocks, 2, KV heads, 16]
    changed[0, w.tables[0][2], :, :, 0] = False
    assert not bool(changed.any())
    w.close()


# ---- commit ---------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("with_prior", [False, True])
@pytest.mark.parametrize("shape", ["4:2x32", "16:8x128", "5:5x64"])
def test_commit_walks_moves_and_quantises(shape, with_prior, kind):
    ctx = [37, 0, 100, 15, 64, 5]
    parents = [random_tree(40, 1), random_tree(16, 2), 200, [-1, 0, 0, 1, 1, 2, 2, 5], [-1, PAD, 0, PAD, 2, 2, 4], random_tree(256, 3)]
    w = Setup8(shape, kind, ctx, parents, layers=3, seed=8, spread=6)
    rng = random.Random(4)
    draft, target, prior = ([rng.randrange(40) for _ in range(w.N)] for _ in range(3))
    prior = prior[:len(ctx)]
    b = 0
    for s, tree in enumerate(w.parents):  # the model agrees all the way down some branch
        if with_prior:
            prior[s] = draft[b] if s != 3 else 99
        at = 0
        while True:
            kids = [i for i, p in enumerate(tree) if p == at]
            if not kids or (s == 1 and at > 3):
                break
            at = rng.choice(kids)
            target[b + w.parents[s][at]] = draft[b + at]
        b += len(tree)
    codes, e = w.codes.clone(), log2(w.scales).transpose(2, 3).clone()
    values = w.values()
    b = 0
    for s, tree in enumerate(w.parents):
        n = len(tree)
        way = walk(tree, draft[b:b + n], target[b:b + n], prior[s] if with_prior else None)
        for p in range(w.ctx[s] // 16, (w.ctx[s] + len(way) + 15) // 16):
            mine = [(w.ctx[s] + i, w.ctx[s] + x) for i, x in enumerate(way) if (w.ctx[s] + i) // 16 == p]
            going = [(to, frm) for to, frm in mine if to != frm]
            if not going:
                continue
            blk = w.tables[s][p]
            rows = [values[:, w.where(s, frm)[0], :, :, frm % 16] for _, frm in going]  # [layers, 2, KV heads, D]
            new = torch.maximum(e[:, blk], need(torch.stack(rows).abs().amax((0, -1)), kind))
            stay = [r for r in range(16) if p * 16 + r < w.ctx[s]] + [to % 16 for to, frm in mine if to == frm]
            for r in stay:
                codes[:, blk, :, :, r] = codes_of(values[:, blk, :, :, r], new[..., None], kind)
            for (to, _), row in zip(going, rows):
                codes[:, blk, :, :, to % 16] = codes_of(row, new[..., None], kind)
            e[:, blk] = new
        b += n
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    accepted, path, after = w.trees.commit(dev(draft), dev(target), dev(prior) if with_prior else None)
    b = 0
    for s, tree in enumerate(w.parents):
        n = len(tree)
        way = walk(tree, draft[b:b + n], target[b:b + n], prior[s] if with_prior else None)
        assert accepted[s] == len(way) and path[b:b + n].tolist() == way + [-1] * (n - len(way))
        assert after[s] == (target[b + way[-1]] if way else prior[s] if with_prior else -1)
        b += n
    assert torch.equal(log2(w.scales).transpose(2, 3), e)
    assert torch.equal(w.codes, codes)
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", ["4:2x32", "8:4x64", "16:8x128"])
@pytest.mark.parametrize("ctx", [0, 5, 16])
def test_commit_between_pages_of_one_scale_copies_codes(ctx, shape, kind):
    """Every code may move over one that another lane of the warp has to move on: chains that leave out every other node, or
    all but the last ones, over pages of the same scale."""
    step = [i - 2 if i > 1 else i - 1 for i in range(100)]  # 0, 2, 4, .. and 0, 1, 3, 5, ..
    far = [-1] + [0] * 50 + list(range(50, 90))
    w = Setup8(shape, kind, [ctx] * 3, [step, step, far], layers=4, seed=2)
    w.scales[:] = 2.0 ** -4
    ways = [list(range(0, 100, 2)), [0] + list(range(1, 100, 2)), [0] + list(range(50, 91))]
    draft = torch.arange(w.N, dtype=torch.int32, device="cuda")
    target = torch.full((w.N,), -1, dtype=torch.int32)
    want, b = w.codes.clone(), 0
    for s, way in enumerate(ways):
        for x, y in zip(way, way[1:]):
            target[b + x] = b + y
        for i, x in enumerate(way):
            (to, r), (frm, z) = w.where(s, ctx + i), w.where(s, ctx + x)
            want[:, to, :, :, r] = w.codes[:, frm, :, :, z]
        b += len(w.parents[s])
    accepted, _, _ = w.trees.commit(draft, target.cuda())
    assert accepted.tolist() == [len(x) for x in ways]
    assert torch.equal(w.codes, want) and bool((w.scales == 2.0 ** -4).all())
    w.close()


# ---- read -----------------------------------------------------------------------------------------------------


def read_rows(w, part):
    return [(s, slot) for s in range(len(w.ctx)) if w.parents[s] for slot in range(w.ctx[s] // 16 * 16 if part else 0, w.ctx[s] + len(w.parents[s]))]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_read_gives_the_values(batch, shape, kind):
    ctx, parents = BATCHES[batch]
    w = Setup8(shape, kind, ctx, parents, layers=3, seed=len(batch), spread=4)
    values = w.values()
    for part in (dec.DEC_READ_ALL, dec.DEC_READ_PAGES):
        rows = read_rows(w, part)
        at = torch.tensor([w.where(s, x) for s, x in rows], device="cuda").T
        want = values[1:][:, at[0], :, :, at[1]].permute(1, 0, 2, 3, 4)  # [layers, rows, 2, KV heads, D]
        for out_type in (torch.bfloat16, torch.float16, torch.float32):
            k, v = w.trees.read(1, part, out_type, layers=2)
            assert k.shape == (2, len(rows), w.Hkv, w.D)
            assert torch.equal(k, want[:, :, 0].to(out_type)) and torch.equal(v, want[:, :, 1].to(out_type))
        k, _ = w.trees.read(2, part)
        assert torch.equal(k, want[1, :, 0].to(torch.bfloat16))
    w.close()


@pytest.mark.parametrize("cache", ["f16", "f32"])
@pytest.mark.parametrize("shape", ["4:2x32", "8:4x64", "16:8x128"])
def test_read_of_caches_that_are_not_quantised(shape, cache):
    from tests.test_gpu_trees import Setup

    w = Setup(shape, cache, [37, 0, 100, 16], [9, 5, 0, [-1, PAD]], seed=1)
    for part in (dec.DEC_READ_ALL, dec.DEC_READ_PAGES):
        at = torch.tensor([w.where(s, x) for s, x in read_rows(w, part)], device="cuda").T
        want = w.slab[:, at[0], :, :, at[1]].permute(1, 0, 2, 3, 4)
        for out_type in (torch.bfloat16, torch.float16, torch.float32):
            k, v = w.trees.read(0, part, out_type, layers=2)
            assert torch.equal(k, want[:, :, 0].to(out_type)) and torch.equal(v, want[:, :, 1].to(out_type))
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
def test_read_into_given_rows_and_one_side_alone(kind):
    w = Setup8("8:4x64", kind, [37, 5], [9, 5], seed=1)
    k, v = w.trees.read(0, dec.DEC_READ_ALL, torch.float16)
    rows, width = k.shape[0], 4 * 64
    only = torch.full_like(k, 3.0)
    w.trees.read(0, dec.DEC_READ_ALL, out=(only, None))
    assert torch.equal(only, k)
    w.trees.read(0, dec.DEC_READ_ALL, out=(None, only))
    assert torch.equal(only, v)
    # rows further apart than they are wide, at an address that is a multiple of four elements only, two layers
    L, st = dec.lib(), torch.cuda.current_stream().cuda_stream
    both = w.trees.read(0, dec.DEC_READ_ALL, torch.float16, layers=2)
    for ld in (width + 4, width + 8):
        gap = rows * ld + 20
        wide = [torch.full((4 + 2 * gap + 64,), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
        assert L.dec_tree_read(w.trees.handle, 0, 2, 0, rows, dec.DEC_T_F16, *(x.data_ptr() + 8 for x in wide), ld, gap, C.c_void_p(st)) == 0
        for x, want in zip(wide, both):
            for layer in range(2):
                got = x[4 + layer * gap:4 + layer * gap + rows * ld].view(rows, ld)
                assert torch.equal(got[:, :width], want[layer].reshape(rows, width))
                got[:, :width] = 3.0
            assert bool((x == 3.0).all())
    w.close()


def test_rows_past_two_to_the_31_are_refused():
    """Sequences that share a long prompt have more rows than 32 bits count; what they changed is read as ever."""
    seqs, ctx = 53000, 40900  # 2556 shared blocks, slots 4 .. of a block of their own
    H, Hkv, D = SHAPES["4:2x32"]
    shape = {"vocab": 512, "d_model": 64, "n_layers": 1, "n_heads": H, "n_kv_heads": Hkv, "head_dim": D, "ff_hidden": 64}
    shared = ctx // 16
    pool = KvPool(shape, dec.DEC_BF16_F16KV, shared + seqs, max_positions=40960, kv_type=dec.DEC_T_I8)
    ids = torch.tensor(pool.alloc(shared + seqs), dtype=torch.int32)
    table = torch.empty((seqs, shared + 1), dtype=torch.int32)
    table[:, :shared], table[:, shared] = ids[:shared], ids[shared:]
    trees = DraftTrees(pool, seqs, seqs, shared + 1)
    arrays = (torch.arange(seqs + 1, dtype=torch.int32), torch.full((seqs,), ctx, dtype=torch.int32), torch.full((seqs,), -1, dtype=torch.int32), table)
    b = dec.dec_tree_batch(seqs, seqs, *(C.cast(x.data_ptr(), C.POINTER(C.c_int32)) for x in arrays), shared + 1)
    L, st, rows = dec.lib(), C.c_void_p(torch.cuda.current_stream().cuda_stream), C.c_int64(7)
    assert L.dec_tree_set(trees.handle, C.byref(b), st) == dec.DEC_OK
    assert L.dec_tree_read_rows(trees.handle, dec.DEC_READ_ALL, C.byref(rows)) == dec.DEC_ERANGE and rows.value == 7
    out = torch.full((seqs * 5, Hkv, D), 3.0, device="cuda")
    for n in (seqs * 5, seqs * (ctx + 1), (seqs * (ctx + 1) + 2 ** 31) % 2 ** 32 - 2 ** 31):
        assert L.dec_tree_read(trees.handle, 0, 1, dec.DEC_READ_ALL, n, dec.DEC_T_F32, out.data_ptr(), None, Hkv * D, 0, st) == dec.DEC_ERANGE
    trees.n_tokens, trees.n_seqs = seqs, seqs
    assert L.dec_tree_read_rows(trees.handle, dec.DEC_READ_PAGES, C.byref(rows)) == dec.DEC_OK and rows.value == seqs * 5
    k = torch.randn((seqs, Hkv, D), device="cuda")
    trees.append(0, None, k, k)
    assert L.dec_tree_read(trees.handle, 0, 1, dec.DEC_READ_PAGES, seqs * 5, dec.DEC_T_F32, out.data_ptr(), None, Hkv * D, 0, st) == dec.DEC_OK
    got = out.view(seqs, 5, Hkv, D)
    assert not bool(got[:, :4].any()) and float((got[:, 4] - k).abs().max()) <= float(k.abs().max()) / 63 / 2
    assert trees.status() == 0
    trees.close()
    pool.close()


# ---- together, captured, on streams ------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shape", ["8:4x64", "16:8x128"])
def test_steps_of_drafting_give_the_plain_sequence(shape, kind):
    """Append, attend, commit, step after step, against a cache that is kept in 64 bits: what is accepted lies within the
    codes' steps of what was given, and attention is the formula over what is cached."""
    w = Setup8(shape, kind, [0], [1], layers=1, seed=6, extra_blocks=20)
    blocks = w.tables[0] + [b for b in range(w.blocks) if b not in w.tables[0]][:15]
    w.tables = [blocks]
    rng = random.Random(2)
    plain, ctx = [], 0
    rope, freq = RopeTable(w.D, 600), frequencies(w.D, 1e6, dec.DEC_ROPE_PLAIN, 1.0, 0, 0, 0)
    w.trees.close()
    w.trees = DraftTrees(w.pool, 1, 64, 24)
    for step in range(12):
        tree = random_tree([1, 5, 17, 30][step % 4], step)
        w.ctx, w.parents, w.N = [ctx], [tree], len(tree)
        w.trees.set(w.ctx, w.parents, w.tables)
        k, v, q = w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.H, w.D)
        q = w.trees.append(0, q, k, v, rope=rope)
        check(w, w.trees.attend(0, q), 0, q)
        pos = torch.tensor([p for *_, p in w.nodes()], device="cuda")
        kf = formed(k, None, pos, w.D, dec.DEC_ROPE_HALF, freq, 1.0)
        draft = [rng.randrange(1000) for _ in tree]
        target, at = [-1] * w.N, 0
        while [i for i, p in enumerate(tree) if p == at]:
            to = rng.choice([i for i, p in enumerate(tree) if p == at])
            target[at], at = draft[to], to
        way = walk(tree, draft, target, None)
        accepted, _, _ = w.trees.commit(torch.tensor(draft, dtype=torch.int32, device="cuda"), torch.tensor(target, dtype=torch.int32, device="cuda"))
        assert int(accepted) == len(way)
        plain += [(kf[i], v[i].double()) for i in way]
        ctx += len(way)
    w.ctx, w.parents, w.N = [ctx], [[-1]], 1
    w.trees.set(w.ctx, w.parents, w.tables)
    k, v = w.trees.read(0, dec.DEC_READ_ALL, torch.float32)
    sc = torch.stack([w.scales[0, w.where(0, x)[0]].double() for x in range(ctx)])  # [slots, KV heads, 2]
    for got, side in ((k, 0), (v, 1)):
        want = torch.stack([p[side] for p in plain])
        e = sc[:, :, side, None]
        # i8: 1/2 + 1/4 + .. steps; e4m3: half a step of the value, and of subnormal codes as i8; fp32's rounding of a key
        allowed = (e if kind == "i8" else 2.0 ** -4 * want.abs() + 2.0 ** -9 * e) + 2.0 ** -20 * want.abs().amax()
        assert bool(((got[:ctx].double() - want).abs() <= allowed).all())
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
def test_a_rejected_draft_rounds_the_accepted_tokens_of_its_page(kind):
    """What the documents say of it: its scale stays, and the page's tokens keep the bits of that scale only; pages in front
    of it, the same step without that node, and a page that begins anew do not have it."""
    at = {}
    for large in (False, True):
        w = Setup8("16:8x128", kind, [20], [[-1, 0, 0]], seed=3, extra_blocks=1)
        blocks = w.tables[0] + [b for b in range(w.blocks) if b not in w.tables[0]][:1]
        w.tables = [blocks]
        w.trees.close()
        w.trees = DraftTrees(w.pool, 1, 16, 4)
        w.trees.set([20], [[-1, 0, 0]], w.tables)
        x = torch.randn((2, 3, w.Hkv, w.D), generator=w.g).cuda()
        first, e = w.values()[0, blocks[1]].clone(), log2(w.scales[0, blocks[1]]).T
        before = w.codes[0, blocks[0]].clone()
        if large:
            x[:, 1] *= 2.0 ** 12  # node 1 is rejected
        w.trees.append(0, None, x[0], x[1])
        draft, target = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([5, 6, 7], [7, 0, 0]))
        accepted, path, _ = w.trees.commit(draft, target)
        assert accepted.tolist() == [2] and path.tolist() == [0, 2, -1]
        # the next step: one token in the same page, which needs less
        w.trees.set([22], [[-1]], w.tables)
        w.trees.append(0, None, x[0, :1], x[1, :1])
        e_now = log2(w.scales[0, blocks[1]]).T
        want_e = torch.maximum(e, need(x.double().abs().amax((1, 3)), kind))
        assert torch.equal(e_now, want_e) and torch.equal(w.codes[0, blocks[0]], before)
        # cached tokens 16 .. 19: their codes at the scale that the page had, rounded again to what it has now
        now = w.values()[0, blocks[1]]
        assert torch.equal(now[:, :, :4], numbers(codes_of(first[:, :, :4], e_now[..., None, None], kind), kind) * two(e_now)[..., None, None])
        at[large] = float((now[:, :, :4] - first[:, :, :4]).norm() / first[:, :, :4].norm())
        # sixteen chained tokens later the next page has only its own rows' scale
        w.trees.set([23], [10], w.tables)
        y = torch.randn((2, 10, w.Hkv, w.D), generator=w.g).cuda()
        w.trees.append(0, None, y[0], y[1])
        assert torch.equal(log2(w.scales[0, blocks[2]]).T, need(y[:, 9:].double().abs().amax((1, 3)), kind))
        w.close()
    assert at[True] > 16 * at[False]  # seven of i8's eight bits gone, e4m3's small values among its subnormal codes


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("seqs, nodes", [(3, 6), (30, 7), (10, 60), (4, 200)])
def test_captured_calls_follow_the_plan(seqs, nodes, kind):
    total = seqs * nodes
    rng = random.Random(seqs)
    w = Setup8("16:8x128", kind, [40 + 31 * s for s in range(seqs)], [nodes] * seqs, seed=1, extra_blocks=8 * seqs, max_tokens=total)
    q, k, v = w.rand(total, w.H, w.D), w.rand(total, w.Hkv, w.D), w.rand(total, w.Hkv, w.D)
    rope = RopeTable(128, 2000)
    draft = torch.randint(5, (total,), generator=w.g, dtype=torch.int32).cuda()
    target = torch.randint(5, (total,), generator=w.g, dtype=torch.int32).cuda()

    def step(read):
        qr = w.trees.append(0, q, k, v, rope=rope)
        out = w.trees.attend(0, qr)
        got = w.trees.commit(draft, target)
        return (qr, out, *got, *(w.trees.read(0, dec.DEC_READ_PAGES, layers=2) if read else ()))

    step(True)
    torch.cuda.synchronize()
    start = w.buf.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(False)
    pool_ids = [b for b in range(w.blocks)]
    for turn in range(4):
        # the same shape, divided in another way: the first sequence keeps the most nodes, others give some to padding
        ctx = [rng.randrange(0, 120) for _ in range(seqs)]
        parents = [random_tree(nodes, turn * 50 + s) for s in range(seqs)]
        for s in range(1, seqs):
            for i in rng.sample(range(nodes), rng.randrange(0, nodes)):
                if i not in parents[s]:
                    parents[s][i] = PAD
        rng.shuffle(pool_ids)
        need_blocks, at = [(c + nodes + 15) // 16 for c in ctx], 0
        if sum(need_blocks) > w.blocks:
            ctx, need_blocks = [0] * seqs, [(nodes + 15) // 16] * seqs
        tables = []
        for n in need_blocks:
            tables.append(pool_ids[at:at + n])
            at += n
        w.ctx, w.parents, w.tables = ctx, parents, tables
        w.trees.set(ctx, parents, tables)
        w.buf.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in held] + [w.buf.clone()]
        w.buf.copy_(start)
        direct = [*step(False), w.buf]
        assert torch.equal(replayed[0], direct[0])
        # the split's parts may be added in another order
        assert float((replayed[1].float() - direct[1].float()).abs().max()) <= 2.0 ** -6 * max(1.0, float(direct[1].float().abs().max()))
        for x, y in zip(replayed[2:], direct[2:]):
            assert torch.equal(x, y)
    assert w.trees.status() == 0
    w.close()


@pytest.mark.parametrize("kind", ["f16", *KINDS])
@pytest.mark.parametrize("captured, replayed", [(4, 8), (4, 20), (8, 4), (8, 30), (20, 4), (20, 8)])
def test_captured_append_commit_and_read_follow_plans_of_other_attention_kernels(captured, replayed, kind):
    """16 sequences, 64 nodes, one word of mask: the longest sequence decides the attention's kernel and grid, and the other
    calls' replays do not mind."""
    def sizes(longest, seed):
        rng, n = random.Random(seed), [longest] + [1] * 15
        while sum(n) < 64:
            i = rng.randrange(1, 16)
            n[i] += n[i] < longest
        return n

    from tests.test_gpu_trees import Setup

    def trees_of(longest, seed):
        return [random_tree(n, seed * 50 + i) for i, n in enumerate(sizes(longest, seed))]

    ctx = [21 + 9 * s for s in range(16)]
    parents = trees_of(captured, 1)
    w = Setup("16:8x128", "f16", ctx, parents, seed=2, extra_blocks=64) if kind == "f16" else Setup8("16:8x128", kind, ctx, parents, seed=2, extra_blocks=64)
    buf = w.slab if kind == "f16" else w.buf
    q, k, v = w.rand(64, w.H, w.D), w.rand(64, w.Hkv, w.D), w.rand(64, w.Hkv, w.D)
    rope = RopeTable(128, 2000)
    draft, target = (torch.randint(2, (64,), generator=w.g, dtype=torch.int32).cuda() for _ in range(2))

    def step():
        return (w.trees.append(0, q, k, v, rope=rope), *w.trees.commit(draft, target), *w.trees.read(0, layers=2))

    step()
    torch.cuda.synchronize()
    start = buf.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(3):
        parents = trees_of(replayed, turn + 2)
        ctx = list(reversed(ctx))  # as many rows in all
        ids = list(range(w.blocks))
        random.Random(turn).shuffle(ids)
        tables = [[ids.pop() for _ in range((c + len(p) + 15) // 16)] for c, p in zip(ctx, parents)]
        w.trees.set(ctx, parents, tables)
        buf.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        replayed_to = [x.clone() for x in held] + [buf.clone()]
        buf.copy_(start)
        for x, y in zip(replayed_to, [*step(), buf]):
            assert torch.equal(x, y)
    assert w.trees.status() == 0
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
def test_a_captured_read_of_another_number_of_rows_does_nothing(kind):
    w = Setup8("8:4x64", kind, [40, 40], [3, 3], seed=1, extra_blocks=4)
    w.trees.read(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = w.trees.read(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], w.trees.read(0)[0])
    w.trees.set([41, 40], [3, 3], w.tables)
    for x in held:
        x.fill_(5.0)
    graph.replay()
    assert w.trees.status() == dec.DEC_DEV_SHAPE
    assert all(bool((x == 5.0).all()) for x in held)
    w.trees.set([39, 41], [3, 3], w.tables)  # as many rows, divided in another way
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[1], w.trees.read(0)[1])
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("captured, replayed", [([5] * 20, [100]), ([5] * 20, [4] * 25), ([100], [5] * 20), ([60, 40], [100]), ([100], [120]), ([6] * 4, [6] * 5), ([9], [8])])
def test_captured_calls_on_a_plan_of_another_shape_do_nothing(captured, replayed, kind):
    """Sequences, nodes or mask words differ (the attention's rows in the last pair, too)."""
    w = Setup8("16:8x128", kind, [40 + 7 * s for s in range(len(captured))], captured, seed=1, extra_blocks=300, max_tokens=128)
    n, seqs = w.N, len(captured)
    w.trees.close()
    w.trees = DraftTrees(w.pool, 32, 128, 16)
    w.trees.set(w.ctx, w.parents, w.tables)
    q, k, v = w.rand(n, w.H, w.D), w.rand(n, w.Hkv, w.D), w.rand(n, w.Hkv, w.D)
    draft, target = (torch.randint(2, (n,), generator=w.g, dtype=torch.int32).cuda() for _ in range(2))

    def calls():
        return ((w.trees.append(0, q, k, v),), (w.trees.attend(0, q),), w.trees.commit(draft, target), w.trees.read(0))

    calls()
    torch.cuda.synchronize()
    graphs, held = [], []
    for i in range(4):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append((lambda: (w.trees.append(0, q, k, v),), lambda: (w.trees.attend(0, q),), lambda: w.trees.commit(draft, target), lambda: w.trees.read(0))[i]())
    ids = list(range(w.blocks))
    random.Random(1).shuffle(ids)
    ctx = [33 + 5 * s for s in range(len(replayed))]
    tables = [[ids.pop() for _ in range((c + m + 15) // 16)] for c, m in zip(ctx, replayed)]
    w.trees.set(ctx, replayed, tables)
    for graph, out in zip(graphs, held):
        for x in out:
            x.fill_(3)
        start = w.buf.clone()
        graph.replay()
        assert w.trees.status() == dec.DEC_DEV_SHAPE
        assert torch.equal(w.buf, start) and all(bool((x == 3).all()) for x in out)
    w.trees.set(w.ctx, w.parents, w.tables)  # and follow the plan of their capture again
    for graph in graphs:
        graph.replay()
    assert w.trees.status() == 0
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("nodes", [4, 50, 150])
def test_two_plans_on_two_streams(nodes, kind):
    ws = [Setup8("16:8x128", kind, [300, 77], [nodes, nodes], seed=s) for s in range(2)]
    qs = [w.rand(w.N, w.H, w.D) for w in ws]
    kv = [(w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)) for w in ws]
    want = []
    for w, q, (k, v) in zip(ws, qs, kv):
        w.trees.append(0, None, k, v)
        want.append((w.trees.attend(0, q), w.trees.read(0)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ws]
    for _ in range(5):
        got = []
        for w, q, (k, v), st in zip(ws, qs, kv, streams):
            w.trees.append(0, None, k, v, stream=st)
            got.append((w.trees.attend(0, q, stream=st), w.trees.read(0, stream=st)))
        torch.cuda.synchronize()
        for (o, r), (po, pr) in zip(got, want):
            assert torch.equal(o, po) and all(torch.equal(x, y) for x, y in zip(r, pr))
    for w in ws:
        w.close()


def test_pages_past_two_to_the_32_bytes():
    """Blocks behind byte 2^32 of the codes, written, attended and read back."""
    H, Hkv, D = SHAPES["16:8x128"]
    blocks = (1 << 32) // (2 * Hkv * 16 * D) + 40
    shape = {"vocab": 512, "d_model": 64, "n_layers": 1, "n_heads": H, "n_kv_heads": Hkv, "head_dim": D, "ff_hidden": 64}
    pool = KvPool(shape, dec.DEC_BF16_F16KV, blocks, kv_type=dec.DEC_T_I8)
    ids = pool.alloc(blocks)
    table = sorted(ids)[-12:]
    trees = DraftTrees(pool, 1, 180, 12)
    trees.set([0], [180], [table])
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn((180, n, D), generator=g).cuda() for n in (Hkv, Hkv, H))
    trees.append(0, None, k, v)
    gk, gv = trees.read(0, out_type=torch.float32)
    step = k.abs().amax() / 63
    assert float((gk - k).abs().max()) <= step and float((gv - v).abs().max()) <= step
    o = trees.attend(0, q).view(180, H, D).float()
    s = torch.einsum("nhd,khd->nhk", q, gk.repeat_interleave(2, 1)) / math.sqrt(D)
    s = s.masked_fill(torch.ones(180, 180, device="cuda").triu(1).bool()[:, None], -math.inf)
    ref = torch.einsum("nhk,khd->nhd", torch.softmax(s, -1), gv.repeat_interleave(2, 1))
    assert float((o - ref).norm()) <= 2.0 ** -7 * float(ref.norm())
    assert trees.status() == 0
    trees.close()
    pool.close()


def test_refusals():
    w = Setup8("8:4x64", "i8", [40], [3], seed=1)
    L, st, h = dec.lib(), C.c_void_p(torch.cuda.current_stream().cuda_stream), w.trees.handle
    rows, width = 43, 4 * 64
    x = torch.full((2, 2, rows, width), 3.0, device="cuda")
    good = dict(layer=0, n=1, part=0, rows=rows, kind=dec.DEC_T_F32, k=x[0].data_ptr(), v=x[1].data_ptr(), ld=width, stride=0)

    def call(**change):
        a = {**good, **change}
        return L.dec_tree_read(h, a["layer"], a["n"], a["part"], a["rows"], a["kind"], a["k"], a["v"], a["ld"], a["stride"], st)

    for change in ({"layer": 2}, {"layer": -1}, {"n": 0}, {"layer": 1, "n": 2}, {"n": 2}, {"n": 2, "stride": rows * width - 4}, {"n": 2, "stride": rows * width + 2}, {"part": 2}, {"part": -1}, {"rows": 42},
                   {"rows": 44}, {"kind": 3}, {"kind": 7}, {"ld": width - 4}, {"ld": width + 2}, {"k": x[0].data_ptr() + 4}, {"k": None, "v": None}, {"v": x[0].data_ptr()}):
        assert call(**change) == dec.DEC_EINVAL, change
        assert dec.lib().dec_last_error()
    torch.cuda.synchronize()
    assert bool((x == 3.0).all())
    assert call() == dec.DEC_OK
    with pytest.raises(ValueError):
        w.trees.read(0, out=(x[0, 0], None))
    with pytest.raises(ValueError):
        w.trees.read(0, layers=0)
    with pytest.raises(dec.DecError):
        w.trees.read(0, part=5)
    with pytest.raises(dec.DecError):
        w.trees.read(0, out=(None, None))
    q = torch.zeros((3, 8, 64), device="cuda")
    assert L.dec_tree_attend(h, 0, q.data_ptr(), 0, 512, x.data_ptr(), dec.DEC_T_F32, 512, st) == dec.DEC_EINVAL
    ctx, table = (C.c_int32 * 1)(40), (C.c_int32 * 3)(*w.tables[0])
    assert L.dec_attend_noalloc(w.pool.pool, 0, 1, q.data_ptr(), ctx, table, 3, x.data_ptr(), st) == dec.DEC_EINVAL
    w.close()
