"""Block tables of different lengths in one batch (no GPU): a table that ends
before its sequence's last slot is refused, whatever the other tables'
lengths, and one that need not be longer is taken."""

import ctypes as C

import pytest

pytest.importorskip("torch")

from decoder_qwen3_step_gb300 import dec, inputs, trees  # noqa: E402
from decoder_qwen3_step_gb300.runtime import Batch, Decoder, make_config  # noqa: E402


@pytest.fixture()
def pool():
    L = dec.lib()
    cfg = make_config(inputs.SHAPES["tiny"], dec.DEC_FP32, 200)
    size, p = C.c_size_t(), C.c_void_p()
    assert L.dec_pool_bytes(C.byref(cfg), 12, C.byref(size)) == 0
    # host bookkeeping only: the slab address is never read here
    assert L.dec_pool_create(C.byref(cfg), 12, C.c_void_p(1 << 40), size.value, C.byref(p)) == 0
    ids = (C.c_int32 * 12)()
    assert L.dec_pool_alloc(p, 12, ids) == 0  # all of them: block 0 is somebody's
    yield L, p
    L.dec_pool_destroy(p)


@pytest.mark.parametrize("ctx, nodes, tables, taken", [
    ([18, 33], [1, 1], [[5], [6, 7, 8]], False),        # slot 18 lies in a second block that the first table lacks
    ([15, 33], [1, 1], [[5], [6, 7, 8]], True),
    ([15, 33], [2, 1], [[5], [6, 7, 8]], False),
    ([40, 33], [1, 1], [[5, 9], [6, 7, 8]], False),     # the block of the new slot
    ([40, 33], [1, 1], [[], [6, 7, 8]], False),
    ([40, 33], [0, 1], [[], [6, 7, 8]], True),          # no nodes: no table
    ([0, 33], [[-1] * 17, 1], [[5], [6, 7, 8]], False),
])
def test_tree_tables(pool, ctx, nodes, tables, taken):
    L, p = pool
    b, keep = trees.tree_batch(ctx, nodes, tables)
    code = L.dec_tree_check(p, C.byref(b))
    assert code == dec.DEC_OK if taken else code in (dec.DEC_EBLOCK, dec.DEC_ERANGE)


@pytest.mark.parametrize("seqs, taken", [
    ([([1], 18, [5]), ([1], 33, [6, 7, 8])], False),
    ([([1], 15, [5]), ([1], 33, [6, 7, 8])], True),
    ([([1, 2], 15, [5]), ([1], 33, [6, 7, 8])], False),
    ([([1] * 20, 0, [5, 9]), ([1] * 48, 0, [6, 7, 8])], True),
    ([([1] * 33, 0, [5, 9]), ([1] * 48, 0, [6, 7, 8])], False),
    ([([1], 40, []), ([1], 33, [6, 7, 8])], False),
])
def test_step_tables(pool, seqs, taken):
    """Decoder.prefill and Decoder.decode marshal their step through Batch(...).checked()."""
    L, p = pool
    if taken:
        assert L.dec_batch_check(p, C.byref(Batch(seqs).checked().struct), 0) == dec.DEC_OK
    else:
        with pytest.raises(ValueError):
            Batch(seqs).checked()


def test_a_decoder_refuses_short_tables():
    class Library:
        def __getattr__(self, name):
            raise AssertionError(f"{name} called")

    m = Decoder.__new__(Decoder)
    m.L, m.pool, m.handle = Library(), None, None
    for step in (m.prefill, m.decode):
        with pytest.raises(ValueError):
            step([([1], 18, [5]), ([1], 33, [6, 7, 8])])
