"""Draft trees over inputs that are not finite: a query or key that is NaN
shows in every row that it belongs to, and nowhere else."""

import random

import pytest

torch = pytest.importorskip("torch")

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
