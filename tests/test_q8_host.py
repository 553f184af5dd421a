"""A pool held in 8 bits without a GPU: sizes, the layout of codes and scales,
what is refused, and the codes that the tests of the kernels go by."""

import ctypes as C

import pytest

from decoder_qwen3_step_gb300 import dec, inputs
from decoder_qwen3_step_gb300.runtime import make_config

torch = pytest.importorskip("torch")

from tests.q8_reference import codes_of, need, numbers, rounded  # noqa: E402


def config(name="tiny", mode=dec.DEC_BF16_F16KV, **change):
    c = make_config(inputs.SHAPES[name], mode, 200)
    for k, v in change.items():
        setattr(c, k, v)
    return c


def create(cfg, kind, n, short=0, at=1 << 40):
    L, size, p = dec.lib(), C.c_size_t(), C.c_void_p()
    rc = L.dec_pool_q8_bytes(C.byref(cfg), kind, n, C.byref(size))
    # host bookkeeping only: the slab address is never read here
    return (rc or L.dec_pool_q8_create(C.byref(cfg), kind, n, C.c_void_p(at) if at else None, size.value - short, C.byref(p))), size.value, p


@pytest.mark.parametrize("kind", [dec.DEC_T_E4M3, dec.DEC_T_I8])
@pytest.mark.parametrize("name", ["tiny", "small", "qwen3_0p6b"])
def test_sizes_and_layout(name, kind):
    L, cfg, n = dec.lib(), config(name), 7
    rc, size, p = create(cfg, kind, n)
    assert rc == dec.DEC_OK
    pages = cfg.n_layers * n * 2 * cfg.n_kv_heads
    scales = (pages * 16 * cfg.head_dim + 255) // 256 * 256
    assert size == scales + 4 * pages
    table, at = (C.c_int32 * 2)(5, 3), C.c_int64()
    seen = set()
    for layer in range(cfg.n_layers):
        for head in range(cfg.n_kv_heads):
            for is_v in (0, 1):
                assert L.dec_kv_scale_offset(p, table, 2, 17, layer, head, is_v, C.byref(at)) == 0
                assert at.value == scales + 4 * (((layer * n + 3) * cfg.n_kv_heads + head) * 2 + is_v)
                seen.add(at.value)
                assert L.dec_kv_offset(p, table, 2, 17, layer, head, is_v, C.byref(at)) == 0
                assert at.value == (((layer * n + 3) * 2 + is_v) * cfg.n_kv_heads + head) * 16 * cfg.head_dim + cfg.head_dim
    assert len(seen) == cfg.n_layers * cfg.n_kv_heads * 2 and max(seen) < size
    for args, code in (((17, 0, 0, 2), dec.DEC_EINVAL), ((17, 0, cfg.n_kv_heads, 0), dec.DEC_EINVAL), ((17, cfg.n_layers, 0, 0), dec.DEC_EINVAL), ((32, 0, 0, 0), dec.DEC_ERANGE), ((-1, 0, 0, 0), dec.DEC_EINVAL)):
        pos, layer, head, is_v = args
        assert L.dec_kv_scale_offset(p, table, 2, pos, layer, head, is_v, C.byref(at)) == code
    assert L.dec_kv_scale_offset(p, table, 2, 17, 0, 0, 0, None) == dec.DEC_EINVAL
    assert L.dec_kv_scale_offset(None, table, 2, 17, 0, 0, 0, C.byref(at)) == dec.DEC_EINVAL
    L.dec_pool_destroy(p)


def test_refusals():
    L = dec.lib()
    for kind in (dec.DEC_T_F32, dec.DEC_T_F16, dec.DEC_T_BF16, 5, -1):
        assert create(config(), kind, 4)[0] == dec.DEC_EINVAL
    assert create(config(mode=dec.DEC_FP32), dec.DEC_T_I8, 4)[0] == dec.DEC_EINVAL
    assert create(config(head_dim=96), dec.DEC_T_I8, 4)[0] == dec.DEC_EINVAL
    assert create(config(), dec.DEC_T_I8, 0)[0] == dec.DEC_EINVAL
    assert create(config(), dec.DEC_T_I8, -3)[0] == dec.DEC_EINVAL
    assert create(config(), dec.DEC_T_I8, 4, short=1)[0] == dec.DEC_EINVAL
    assert create(config(), dec.DEC_T_I8, 4, at=(1 << 40) + 16)[0] == dec.DEC_EINVAL
    assert create(config(), dec.DEC_T_I8, 4, at=0)[0] == dec.DEC_EINVAL
    cfg = config()
    assert L.dec_pool_q8_bytes(C.byref(cfg), dec.DEC_T_I8, 4, None) == dec.DEC_EINVAL
    # the pools that have no scales
    size, p, table, at = C.c_size_t(), C.c_void_p(), (C.c_int32 * 1)(0), C.c_int64()
    assert L.dec_pool_bytes(C.byref(cfg), 4, C.byref(size)) == 0
    assert L.dec_pool_create(C.byref(cfg), 4, C.c_void_p(1 << 40), size.value, C.byref(p)) == 0
    assert L.dec_kv_scale_offset(p, table, 1, 3, 0, 0, 0, C.byref(at)) == dec.DEC_EINVAL
    L.dec_pool_destroy(p)


def test_bookkeeping_and_trees_are_those_of_any_pool_and_the_decoder_refuses_it():
    from decoder_qwen3_step_gb300.runtime import Batch
    from decoder_qwen3_step_gb300.trees import tree_batch

    L = dec.lib()
    rc, _, p = create(config(), dec.DEC_T_I8, 6)
    assert rc == 0
    ids = (C.c_int32 * 4)()
    assert L.dec_pool_alloc(p, 4, ids) == 0 and L.dec_pool_alloc(p, 3, ids) == dec.DEC_ECAPACITY
    b, keep = tree_batch([20], [5], [list(ids)])
    assert L.dec_tree_check(p, C.byref(b)) == 0
    L.dec_pool_retain(p, ids[1])
    assert L.dec_tree_check(p, C.byref(b)) == dec.DEC_EBLOCK
    step = Batch([([1], 3, list(ids))])
    assert L.dec_batch_check(p, C.byref(step.struct), 1) == dec.DEC_EINVAL
    assert b"8 bits" in L.dec_last_error()
    L.dec_pool_destroy(p)


def test_the_codes_of_the_references():
    """By hand: ties to even, both ends, subnormal e4m3 numbers, exponents at their borders."""
    x = lambda *v: torch.tensor(v, dtype=torch.float64)  # noqa: E731
    assert rounded(x(0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.4, 300.0), "i8").tolist() == [0, 2, 2, 0, -2, 126, 127, 127]
    # e4m3: 8 steps between powers of two; 17 is a tie of 16 and 18, 19 of 18 and 20; 2^-10 of 0 and 2^-9
    assert rounded(x(17, 19, 433, 464, 1000, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 0.0), "e4m3").tolist() == [
        16, 20, 448, 448, 448, -1.0, 0.0, 2.0 ** -8, 2.0 ** -9, 0.0]
    assert need(x(0, 127, 127.0001, 254, 1, 0.9921875, 1e30, 1e-30), "i8").tolist() == [-40, 0, 1, 1, -6, -7, 40, -40]
    assert need(x(0, 448, 448.001, 1, 0.875, 1e30), "e4m3").tolist() == [-40, 0, 1, -8, -9, 40]
    for kind, top in (("i8", 127), ("e4m3", 448)):
        v = x(-top, top, 0, 5)
        assert numbers(codes_of(v * 4, x(2), kind), kind).tolist() == v.tolist()
    every = torch.arange(256, dtype=torch.uint8)
    keep = (every & 0x7F) != 0x7F
    assert torch.equal(codes_of(numbers(every[keep], "e4m3"), x(0), "e4m3"), every[keep])


def test_a_step_that_reads_nothing_back_asks_for_no_rows():
    """set makes one call of the library; the first read of a plan asks for its rows, the next ones do not."""
    from decoder_qwen3_step_gb300.trees import DraftTrees

    calls = []

    class Library:
        def dec_tree_set(self, *_):
            calls.append("set")
            return 0

        def dec_tree_read_rows(self, _, part, n):
            calls.append(("rows", part))
            n._obj.value = 5 + part
            return 0

        def dec_tree_destroy(self, _):
            pass

    class Pool:
        pool = True

    t = DraftTrees.__new__(DraftTrees)
    t.L, t.pool, t.handle, t._read_of = Library(), Pool(), None, {}
    t._kv_heads, t._dim, t._kv_width, t._index, t.device = 2, 32, 64, 0, "cpu"
    t._stream = lambda stream: 0
    t._read = lambda handle, layer, n, part, rows, *rest: calls.append(("read", rows)) and 0
    t.set([3], [2], [[0]])
    assert calls == ["set"]
    for part in (0, 0, 1, 1):
        k, v = t.read(0, part)
        assert k.shape == v.shape == (5 + part, 2, 32)
    assert calls[1:] == [("rows", 0), ("read", 5), ("read", 5), ("rows", 1), ("read", 6), ("read", 6)]
    t.set([3], [2], [[0]])
    t.read(0)
    assert calls[7:] == ["set", ("rows", 0), ("read", 5)]
