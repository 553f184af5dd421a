"""Draft trees at the ends of what attention's weights hold: scores of any size, pages of an 8-bit cache whose scales lie
some powers of two apart."""

import math

import pytest

torch = pytest.importorskip("torch")

from tests.q8_reference import KINDS, codes_of  # noqa: E402
from tests.test_gpu_q8 import Setup8, check  # noqa: E402
from tests.test_gpu_trees import Setup  # noqa: E402

pytestmark = pytest.mark.gpu


def code(x, kind):
    return codes_of(torch.tensor(float(x), dtype=torch.float64), torch.tensor(0.0), kind).item()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("gap", [3, 5, 8, 9, 12])
@pytest.mark.parametrize("shape, seqs, nodes", [("8:4x64", 16, 30), ("16:8x128", 16, 20), ("8:4x64", 8, 200), ("16:8x128", 8, 70), ("16:8x128", 8, 4)])
def test_many_small_weights_beside_a_page_of_larger_values(shape, seqs, nodes, gap, kind):
    """Each of the first two tiles has one key with the largest score and a page that nobody looks at, its values 2^gap times
    the others'; all other keys weigh 2^-15.5 of the largest each, which is no whole number of f16's smallest steps."""
    ctx = 4000
    w = Setup8(shape, kind, [ctx] * seqs, [[-1] * nodes] * seqs, layers=1, seed=gap)
    w.scales[:] = 1.0
    low, base, top = code(-64, kind), code(32, kind), code(64, kind)
    w.codes[0, :, 0, :, :, 0] = base
    w.codes[0, :, 1] = code(96, kind)
    for s in range(seqs):
        for tile in range(2):
            b, r = w.where(s, tile * 128 + 40 + tile)
            w.codes[0, b, 0, :, r, 0] = top
            w.codes[0, b, 1, :, r] = code(-96, kind)
            b, _ = w.where(s, tile * 128 + 80)
            w.codes[0, b, 0, :, :, 0] = low
            w.scales[0, b, :, 1] = 2.0 ** gap
        for slot in range(ctx, ctx + nodes):
            b, r = w.where(s, slot)
            w.codes[0, b, 0, :, r, 0] = low
    # exact in f16, as are the codes, so the scores are the formula's but for fp32
    q0 = round(15.474 * math.sqrt(w.D) / 32 * math.log(2) * 256) / 256
    q = torch.zeros((w.N, w.H, w.D), device="cuda")
    q[..., 0] = q0
    small, n = math.exp(-32 * q0 / math.sqrt(w.D)), ctx - 2 * 17
    want = 96 * (n * small - 2) / (n * small + 2)  # what nobody looks at weighs 2^-30 in all
    got = w.trees.attend(0, q, out_type=torch.float16).double()
    # weights: half a step of f16 each, and of its subnormal numbers (2^-25 of a reference that is at most the largest);
    # fp32: scores below 2^5 off by 3 half steps, 72 more for sums and the exponential; then the output's half step
    allowed = 96 * (2.0 ** -11 + n * 2.0 ** -25 / (2 + n * small) + (3 * 32 + 72) * 2.0 ** -24) + 2.0 ** -11 * abs(want)
    assert float((got - want).abs().max()) <= allowed
    w.close()


@pytest.mark.parametrize("gap", [20, 22, 23, 29, 30, 32, 44])
@pytest.mark.parametrize("shape, nodes", [("8:4x64", 60), ("16:8x128", 40), ("16:8x128", 200), ("8:4x64", 256), ("16:8x128", 5), ("4:2x32", 60)])
@pytest.mark.parametrize("kind, fine", [("i8", False), ("e4m3", False), ("e4m3", True)])
def test_keys_beside_a_page_of_far_larger_ones(kind, fine, shape, nodes, gap):
    """Keys of a tile keep their bits whatever the scale of a page next to them, of nodes that the rows do not see; fine:
    keys that are e4m3's smallest numbers."""
    w = Setup8(shape, kind, [112], [[-1] * nodes], layers=1, seed=gap)
    q = w.rand(w.N, w.H, w.D)
    if fine:
        k = w.codes[0, :, 0]
        w.codes[0, :, 0] = torch.where(k & 0x7F != 0, (k & 0x87) | 1, k)  # up to 7 of the steps of 2^-9
        q *= 2.0 ** 20
    b, _ = w.where(0, 112)  # slots 112 .. 127 of the tile 0 .. 127: the first sixteen nodes
    w.scales[0, :, :, 0] = 2.0 ** (-6 if fine else -9 if kind == "i8" else -10)
    w.scales[0, b, :, 0] *= 2.0 ** gap
    out = w.trees.attend(0, q)
    check(w, out, 0, q, set(range(min(16, nodes - 1), w.N, max(w.N // 24, 1))) | {w.N - 1} if nodes > 16 else None)
    w.close()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("values", [-38, 0, 34])
@pytest.mark.parametrize("size", [1e8, 1e9, 1e15])
@pytest.mark.parametrize("shape, nodes", [("8:4x64", 5), ("16:8x128", 3), ("16:8x128", 8), ("16:8x128", 40), ("8:4x64", 200)])
def test_scores_past_the_last_place_of_a_values_exponent(shape, nodes, size, values, kind):
    """Queries so large that one key takes all the weight and its score has no bits left for the exponent of a value's scale:
    the output is that key's value."""
    w = Setup8(shape, kind, [250, 40], [nodes, nodes], layers=1, seed=3)
    w.scales[..., 1] *= 2.0 ** values
    w.scales.clamp_(2.0 ** -40, 2.0 ** 40)
    q = w.rand(w.N, w.H, w.D) * size
    out = w.trees.attend(0, q).view(w.N, w.H, w.D).double()
    assert bool(torch.isfinite(out).all())
    G, rows = w.H // w.Hkv, 0
    for n, s, i, _, _ in w.nodes():
        k, v, _, _ = (x.repeat_interleave(G, 1) for x in w.rows(0, s, w.seen(s, i)))
        sc = torch.einsum("hd,khd->hk", q[n].double(), k) / math.sqrt(w.D)
        size_of = torch.einsum("hd,khd->hk", q[n].double().abs(), k.abs()) / math.sqrt(w.D)
        first = sc.topk(2, -1)
        # f16 queries: half a step of each product (2^-11) on both sides, and 100 so that nothing else weighs anything
        clear = first.values[:, 0] - first.values[:, 1] > 2 * 2.0 ** -11 * 1.01 * size_of.amax(-1) + 100
        for h in clear.nonzero()[:, 0].tolist():
            want = v[first.indices[h, 0], h]
            assert bool(((out[n, h] - want).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) * want.abs()).all()), (n, h)
            rows += 1
    assert rows > w.N
    w.close()


@pytest.mark.parametrize("cache", ["f16", *KINDS])
@pytest.mark.parametrize("blocks", [4, 8, 16])  # a warp of the narrow kernels, a group of a wide unit, of a narrow one meet every such block
@pytest.mark.parametrize("shape, nodes", [("8:4x64", 3), ("16:8x128", 8), ("16:8x128", 40), ("16:8x128", 100)])
def test_scores_whose_last_place_is_sixteen(shape, nodes, blocks, cache):
    """Scores of 2^27 .. 2^28 (in units of log 2) that rise by single last places: a reference and 8 round to the next one."""
    ctx = [16 * blocks * 15] * 20
    w = Setup(shape, "f16", ctx, [[-1] * nodes] * 20, layers=1, seed=1) if cache == "f16" else Setup8(shape, cache, ctx, [[-1] * nodes] * 20, layers=1, seed=1)
    k = torch.zeros((w.blocks, w.Hkv, 16, w.D), dtype=torch.float64, device="cuda")
    k[..., 0] = 96.0
    for s in range(20):
        for slot in range(0, w.ctx[s] + nodes, 16):
            k[w.where(s, slot)[0], ..., 1] = float(slot // 16 // blocks)  # up to 16: exact in all
    if cache == "f16":
        w.slab[0, :, 0] = k.half()
        values = w.slab[0, :, 1]
    else:
        w.codes[0, :, 0] = codes_of(k, torch.zeros((), dtype=torch.float64, device="cuda"), cache)
        w.scales[:] = 1.0
        values = w.values()[0, :, 1]
    q = torch.zeros((w.N, w.H, w.D), device="cuda")
    # 96 q0 log2(e) / sqrt(D) of 2^27 .. 2^28, its last place 16; the second channel adds one of them every `blocks` blocks
    q[..., 0] = 2.0 ** 27 * math.sqrt(w.D) * math.log(2) / 96 * (1.05 + 0.9 * torch.rand(q[..., 0].shape, generator=w.g).cuda())
    q[..., 1] = 16 * math.sqrt(w.D) * math.log(2)
    out = w.trees.attend(0, q).double()
    assert bool(torch.isfinite(out).all())
    assert bool((out.abs() <= values.double().abs().amax() * 1.01).all())
    w.close()
