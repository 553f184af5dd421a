"""Draft trees over inputs that are not finite: a query or key that is NaN
shows in every row that it belongs to, and nowhere else; what append does not
turn it copies."""

import random

import pytest

torch = pytest.importorskip("torch")

from decoder_qwen3_step_gb300 import dec  # noqa: E402
from decoder_qwen3_step_gb300.trees import RopeTable  # noqa: E402

from .test_gpu_trees import Setup, check, random_tree  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache, shape, seqs, nodes, ctx", [
    ("f16", "16:8x128", 2, 7, 100), ("f16", "16:8x128", 1, 6, 3000), ("f16", "16:8x128", 32, 8, 1100),  # up to 16 rows: whole units, many parts, two parts
    ("f16", "8:4x64", 3, 5, 40), ("f16", "4:2x32", 2, 40, 300), ("f16", "4:2x32", 1, 8, 2000),
    ("f16", "16:8x128", 2, 40, 700), ("f16", "16:8x128", 2, 200, 700), ("f32", "8:4x64", 2, 9, 700)])
def test_queries_that_are_nan_give_nan(cache, shape, seqs, nodes, ctx):
    w = Setup(shape, cache, [ctx + 3 * i for i in range(seqs)], [random_tree(nodes, i) for i in range(seqs)], seed=4)
    q = w.rand(w.N, w.H, w.D)
    whole, part = 1, w.N - 2  # a row of NaN, and one NaN among a row's channels
    q[whole] = float("nan")
    q[part, :, 5] = float("nan")
    out = w.trees.attend(0, q)
    assert bool(torch.isnan(out[[whole, part]]).all())
    rest = [n for n in range(w.N) if n not in (whole, part)]
    check(w, out, 0, q, sorted(random.Random(3).sample(rest, min(len(rest), 40))))
    w.close()


@pytest.mark.parametrize("cache", ["f16", "f32"])
@pytest.mark.parametrize("nodes", [4, 40])
def test_a_root_with_nothing_cached_whose_key_is_nan(nodes, cache):
    """The root's only score is NaN, so is every descendant's sum; a second root's rows are not."""
    tree = [-1] + [0] * (nodes - 3) + [-1, nodes - 2]
    w = Setup("16:8x128", cache, [0, 20], [tree, 3], seed=2)
    q = w.rand(w.N, w.H, w.D)
    b, r = w.where(0, 0)
    w.slab[0, b, 0, :, r] = float("nan")
    out = w.trees.attend(0, q)
    assert bool(torch.isnan(out[: nodes - 2]).all())
    check(w, out, 0, q, list(range(nodes - 2, w.N)))
    w.close()


@pytest.mark.parametrize("layout", [dec.DEC_ROPE_HALF, dec.DEC_ROPE_INTERLEAVED])
@pytest.mark.parametrize("shape, rot, cache, nodes", [("8:4x64", 32, "f16", 9), ("16:8x128", 72, "f32", 9), ("16:8x128", 64, "f16", 256), ("4:2x32", 8, "f32", 30)])
def test_channels_that_are_not_turned_are_copied(shape, rot, cache, nodes, layout):
    """A value, or a channel behind rot, that is not finite stays alone in its channel; a turned one reaches its pair."""
    w = Setup(shape, cache, [20, 5], [random_tree(nodes, 1), 3], seed=1)
    q, k, v = w.rand(w.N, w.H, w.D), w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    rope = RopeTable(rot, 400, layout=layout)
    clean = w.trees.append(0, q, k, v, rope=rope)
    odd = (float("nan"), float("inf"), -float("inf"))
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    for i in range(w.N):
        if rot < w.D:
            for x in (q2, k2):
                x[i, :, rot + (3 * i) % (w.D - rot)] = odd[i % 3]
        v2[i, :, (5 * i) % w.D] = odd[i % 3]
    turned = 2, 3  # a node and one of its turned channels
    q2[turned[0], :, turned[1]] = float("inf")
    pair = {turned[1], turned[1] + rot // 2 if layout == dec.DEC_ROPE_HALF else turned[1] - 1}
    got = w.trees.append(1, q2, k2, v2, rope=rope)

    def same(a, b):
        return bool((torch.isnan(a) == torch.isnan(b)).all()) and torch.equal(torch.nan_to_num(a, nan=0.5), torch.nan_to_num(b, nan=0.5))

    want = clean.clone()
    want[..., rot:] = q2[..., rot:]
    others = [c for c in range(w.D) if c not in pair]
    assert same(got[..., others], want[..., others])
    rows = [i for i in range(w.N) if i != turned[0]]
    assert same(got[rows], want[rows]) and not bool(torch.isfinite(got[turned[0]][:, sorted(pair)]).any())
    for n, s, i, slot, pos in w.nodes():
        b, r = w.where(s, slot)
        assert same(w.slab[1, b, 0, :, r, :rot], w.slab[0, b, 0, :, r, :rot])
        assert same(w.slab[1, b, 0, :, r, rot:], k2[n, :, rot:].to(w.cache))
        assert same(w.slab[1, b, 1, :, r], v2[n].to(w.cache))
    w.close()


@pytest.mark.parametrize("cache, nodes", [("f16", 4), ("f16", 40), ("f16", 200), ("f32", 4)])
def test_scores_that_are_all_minus_infinity_give_zeros(cache, nodes):
    w = Setup("16:8x128", cache, [0, 30], [random_tree(nodes, 1), 2], seed=2)
    q = w.rand(w.N, w.H, w.D)
    b, r = w.where(0, 0)
    w.slab[0, b, 0, :, r, 5] = -1.0  # the root's key, the only one that it sees
    q[0, :, 5] = float("inf")
    out = w.trees.attend(0, q)
    assert not bool(out[0].any())
    check(w, out, 0, q, sorted(random.Random(3).sample(range(1, w.N), min(w.N - 1, 30))))
    w.close()
