"""Draft trees without a GPU: what dec_tree_check refuses, the rotary
parameters that are refused, and the marshalling of a batch."""

import ctypes as C

import numpy as np
import pytest

from decoder_qwen3_step_gb300 import dec, inputs
from decoder_qwen3_step_gb300.runtime import make_config

trees = pytest.importorskip("decoder_qwen3_step_gb300.trees")


@pytest.fixture()
def pool():
    L = dec.lib()
    cfg = make_config(inputs.SHAPES["tiny"], dec.DEC_FP32, 200)
    size, p = C.c_size_t(), C.c_void_p()
    assert L.dec_pool_bytes(C.byref(cfg), 40, C.byref(size)) == 0
    # host bookkeeping only: the slab address is never read here
    assert L.dec_pool_create(C.byref(cfg), 40, C.c_void_p(1 << 40), size.value, C.byref(p)) == 0
    yield L, p
    L.dec_pool_destroy(p)


def blocks(L, p, n):
    ids = (C.c_int32 * n)()
    assert L.dec_pool_alloc(p, n, ids) == 0
    return list(ids)


def check(L, p, ctx, parents, tables, change=None):
    b, keep = trees.tree_batch(ctx, parents, tables)
    for k, v in (change or {}).items():
        setattr(b, k, v)
    return L.dec_tree_check(p, C.byref(b))


def test_trees_that_are_taken(pool):
    L, p = pool
    t = [blocks(L, p, 3), blocks(L, p, 1), blocks(L, p, 17)]
    assert check(L, p, [33], [5], [t[0]]) == dec.DEC_OK
    assert check(L, p, [0, 33], [1, [-1, 0, 0, 1, -1, dec.DEC_TREE_PAD]], [t[1], t[0]]) == dec.DEC_OK
    assert check(L, p, [9, 5, 0], [0, 7, 16], [[], t[0], t[1]]) == dec.DEC_OK  # a sequence without nodes needs no table
    # the widest tree: 256 nodes at depths far below the end of the positions
    assert check(L, p, [10], [[-1] + [0] * 255], [t[2]]) == dec.DEC_OK


@pytest.mark.parametrize("code, ctx, parents, tables", [
    (dec.DEC_EINVAL, [], [], []),                                   # no sequences
    (dec.DEC_EINVAL, [4], [0], [[0]]),                              # no nodes
    (dec.DEC_EINVAL, [4], [[-1, 1]], [[0]]),                        # a node as its own parent
    (dec.DEC_EINVAL, [4], [[-1, 2, 0]], [[0]]),                     # a later node as parent
    (dec.DEC_EINVAL, [4], [[-3]], [[0]]),                           # neither root nor padding
    (dec.DEC_EINVAL, [4], [[-1, -2, 1]], [[0]]),                    # a child of padding
    (dec.DEC_ERANGE, [-1], [1], [[0]]),                             # a negative context
    (dec.DEC_ERANGE, [201], [1], [list(range(13))]),                # past max_positions
    (dec.DEC_ERANGE, [199], [2], [list(range(13))]),                # the second node's position is
    (dec.DEC_ERANGE, [0], [257], [list(range(17))]),                # more nodes than a tree may have
    (dec.DEC_ERANGE, [15], [2], [[0]]),                             # slot 16 has no block
    (dec.DEC_EBLOCK, [4], [1], [[40]]),                             # outside the pool
    (dec.DEC_EBLOCK, [4], [1], [[-1]]),
    (dec.DEC_EBLOCK, [4], [1], [[30]]),                             # not allocated
    (dec.DEC_EBLOCK, [20], [1], [[30, 0]]),                         # read, not allocated
    (dec.DEC_EBLOCK, [4, 4], [1, 1], [[0], [0]]),                   # written for two sequences
    (dec.DEC_EBLOCK, [4], [20], [[0, 0]]),                          # written for two slots
])
def test_trees_that_are_refused(pool, code, ctx, parents, tables):
    L, p = pool
    blocks(L, p, 20)  # ids 0 .. 19 in some order
    assert check(L, p, ctx, parents, tables) == code
    assert L.dec_last_error()


def test_shared_and_cached_blocks_are_read_but_not_written(pool):
    L, p = pool
    a, b, c = blocks(L, p, 3)
    L.dec_pool_retain(p, a)
    assert check(L, p, [16], [4], [[a, b]]) == dec.DEC_OK
    assert check(L, p, [15], [4], [[a, b]]) == dec.DEC_EBLOCK
    ok = C.c_int32()
    L.dec_pool_set_fill(p, c, 16)
    assert L.dec_pool_register(p, c, 77, C.byref(ok)) == 0 and ok.value == 1
    assert check(L, p, [16], [4], [[c, b]]) == dec.DEC_OK
    assert check(L, p, [3], [4], [[c]]) == dec.DEC_EBLOCK


def test_null_and_crooked_arrays_are_refused(pool):
    L, p = pool
    t = blocks(L, p, 2)
    assert L.dec_tree_check(p, None) == dec.DEC_EINVAL
    assert L.dec_tree_check(None, None) == dec.DEC_EINVAL
    for field in ("seq_start", "ctx", "block_table"):
        assert check(L, p, [4], [3], [t], {field: None}) == dec.DEC_EINVAL, field
    assert check(L, p, [4], [3], [t], {"parents": None}) == dec.DEC_OK  # chains
    assert check(L, p, [4], [3], [t], {"n_tokens": 2}) == dec.DEC_EINVAL
    assert check(L, p, [4], [3], [t], {"max_blocks": 0}) == dec.DEC_EINVAL
    for start in ([1, 3], [0, 5, 3], [0, -1, 3]):
        arr = np.asarray(start, dtype=np.int32)
        b, keep = trees.tree_batch([4] * (len(start) - 1), [3] + [0] * (len(start) - 2), [t] * (len(start) - 1))
        b.seq_start = arr.ctypes.data_as(C.POINTER(C.c_int32))
        assert L.dec_tree_check(p, C.byref(b)) == dec.DEC_EINVAL, start


GOOD = dict(rot_dim=64, layout=0, scaling=0, orig_positions=4096, base=1e4, factor=2.0, low=1.0, high=32.0, attn_factor=1.0)


@pytest.mark.parametrize("change", [
    {"rot_dim": 0}, {"rot_dim": 4}, {"rot_dim": 60}, {"rot_dim": 136}, {"rot_dim": -8}, {"layout": 2}, {"scaling": 4}, {"base": 1.0},
    {"base": float("inf")}, {"base": float("nan")}, {"attn_factor": 0.0}, {"scaling": 1, "factor": 0.5}, {"scaling": 2, "orig_positions": 0},
    {"scaling": 2, "low": 0.0}, {"scaling": 3, "high": 1.0}, {"scaling": 3, "high": float("nan")},
])
def test_rotary_parameters_that_are_refused(change):
    L, size = dec.lib(), C.c_size_t()
    r = dec.dec_rope(**{**GOOD, **change})
    assert L.dec_rope_table_bytes(C.byref(r), 100, C.byref(size)) == dec.DEC_EINVAL
    assert L.dec_last_error()


def test_rotary_table_sizes():
    L, size = dec.lib(), C.c_size_t()
    r = dec.dec_rope(**GOOD)
    assert L.dec_rope_table_bytes(C.byref(r), 100, C.byref(size)) == 0 and size.value == 100 * 32 * 8
    for n in (0, -1, 40961):
        assert L.dec_rope_table_bytes(C.byref(r), n, C.byref(size)) == dec.DEC_ERANGE
    assert L.dec_rope_table_bytes(C.byref(r), 100, None) == dec.DEC_EINVAL
    assert L.dec_rope_table(C.byref(r), 100, C.cast(1 << 40, C.c_void_p), 100, None) == dec.DEC_EINVAL  # too small
    assert L.dec_rope_table(C.byref(r), 100, C.cast((1 << 40) + 4, C.c_void_p), 1 << 20, None) == dec.DEC_EINVAL


def test_calls_without_a_plan_are_refused():
    L = dec.lib()
    x = dec.dec_tree_qkv()
    assert L.dec_tree_append(None, 0, C.byref(x), None) == dec.DEC_EINVAL
    assert L.dec_tree_attend(None, 0, None, 0, 0, None, 0, 0, None) == dec.DEC_EINVAL
    assert L.dec_tree_commit(None, None, None, None, None, None, None, None) == dec.DEC_EINVAL
    assert L.dec_tree_set(None, None, None) == dec.DEC_EINVAL
    assert L.dec_tree_status(None, None, None) == dec.DEC_EINVAL
    L.dec_tree_destroy(None)


def test_batch_marshalling():
    b, (start, ctx, flat, tab) = trees.tree_batch([7, 0, 3], [3, [], [-1, 0, 0]], [[4, 5], [], [9]])
    assert (b.n_seqs, b.n_tokens, b.max_blocks) == (3, 6, 2)
    assert start.tolist() == [0, 3, 3, 6] and ctx.tolist() == [7, 0, 3]
    assert flat[:6].tolist() == [-1, 0, 1, -1, 0, 0] and tab.tolist() == [[4, 5], [0, 0], [9, 0]]
    with pytest.raises(ValueError):
        trees.tree_batch([1], [1, 1], [[0]])
