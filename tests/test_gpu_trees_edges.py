"""Draft trees where calls meet: a wait that has run out and the calls behind
it, streams that order the plan's memory, replays over other trees."""

import ctypes as C

import pytest

torch = pytest.importorskip("torch")

from decoder_qwen3_step_gb300 import dec  # noqa: E402
from decoder_qwen3_step_gb300.trees import DraftTrees, KvPool, RopeTable, tree_batch  # noqa: E402

from .test_gpu_trees import Setup, check, random_tree  # noqa: E402

pytestmark = pytest.mark.gpu


def test_a_part_that_comes_too_late_is_not_taken_for_the_next_calls():
    """30 x 50 nodes: units that the CTAs starting them join.  A wait that runs out is reported, and what comes
    after it leaves no trace for the next call."""
    w = Setup("16:8x128", "f16", [900 + 3 * i for i in range(30)], [random_tree(50, i) for i in range(30)], seed=4)
    L, t = w.trees.L, w.trees
    q = w.rand(w.N, w.H, w.D)
    clean = t.attend(0, q).clone()
    left = C.c_int32(7)
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    for late in (0, 1, 0, 1, 1):
        assert L.dec_debug_tree_join(t.handle, late, 200_000 if late else 1_000_000_000, C.byref(left), stream) == dec.DEC_OK
        assert left.value == 0
        assert t.status() == (dec.DEC_DEV_TIMEOUT if late else 0)
    for layer in (0, 1, 0):
        out = t.attend(layer, q)
    assert torch.equal(out, clean)
    for limit in (0, 999, 1_000_000_001):
        assert L.dec_debug_tree_join(t.handle, 1, limit, C.byref(left), stream) == dec.DEC_EINVAL
    assert L.dec_debug_tree_join(t.handle, 1, 1000, None, stream) == dec.DEC_EINVAL
    w.close()


def test_the_status_belongs_to_the_plan_alone():
    """What an earlier owner of the workspace still writes on the plan's stream is no status of the plan's."""
    w = Setup("8:4x64", "f16", [40], [9], seed=1)
    L, size, h, flags = w.trees.L, C.c_size_t(), C.c_void_p(), C.c_uint32(9)
    assert L.dec_tree_workspace_bytes(w.pool.pool, 1, 9, 8, C.byref(size)) == 0
    buf = torch.zeros(size.value + 256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        buf.fill_(255)  # the earlier owner's last write
    assert L.dec_tree_create(w.pool.pool, 1, 9, 8, C.c_void_p((buf.data_ptr() + 255) & ~255), size.value, C.byref(h)) == 0
    assert L.dec_tree_status(h, C.c_void_p(s.cuda_stream), C.byref(flags)) == 0 and flags.value == 0  # before any call
    b, keep = tree_batch(w.ctx, w.parents, w.tables)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        buf.fill_(255)
    assert L.dec_tree_set(h, C.byref(b), C.c_void_p(s.cuda_stream)) == 0
    q = w.rand(w.N, w.H, w.D)
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty((w.N, w.H * w.D), dtype=torch.bfloat16, device="cuda")
    assert L.dec_tree_attend(h, 0, q.data_ptr(), dec.DEC_T_F32, w.H * w.D, out.data_ptr(), dec.DEC_T_BF16, w.H * w.D, C.c_void_p(s.cuda_stream)) == 0
    assert L.dec_tree_status(h, C.c_void_p(s.cuda_stream), C.byref(flags)) == 0 and flags.value == 0
    assert torch.equal(out, w.trees.attend(0, q))
    L.dec_tree_destroy(h)
    w.close()


def test_tensors_of_calls_on_another_stream_may_be_dropped():
    """Inputs, and a plan with its pool, that are dropped while a call's stream has not come to it yet."""
    w = Setup("16:8x128", "f16", [300, 40], [20, 9], seed=2)
    q, k, v = w.rand(w.N, w.H, w.D), w.rand(w.N, w.Hkv, w.D), w.rand(w.N, w.Hkv, w.D)
    gain = 1 + 0.1 * w.rand(w.D)
    rope = RopeTable(64, 400)
    want_q = w.trees.append(0, q, k, v, rope=rope, q_norm=gain, k_norm=gain)
    want = w.trees.attend(0, want_q).clone()
    draft = torch.arange(w.N, dtype=torch.int32, device="cuda")
    before, blocks, tables, ctx, parents = w.slab.clone(), w.blocks, w.tables, w.ctx, w.parents
    s = torch.cuda.Stream()
    pool = KvPool(w.shape, w.pool.mode, blocks, max_positions=40960, slabs=before)
    pool.alloc(blocks)
    trees = DraftTrees(pool, 2, w.N, 30)
    torch.cuda.synchronize()

    def overwrite(*sizes):
        """Whatever the allocator hands out again is written on the current stream, ahead of s."""
        for n in sizes:
            for _ in range(6):
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)

    sizes = [x.numel() * x.element_size() for x in (q, k, gain, draft, rope.table, before, trees.workspace, want)]
    trees.set(ctx, parents, tables, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    got_q = trees.append(0, q.clone(), k.clone(), v.clone(), rope=RopeTable(64, 400), q_norm=gain.clone(), k_norm=gain.clone(), stream=s)
    got = trees.attend(0, got_q, stream=s)
    copies = [draft.clone(), draft.clone()]
    acc, path, nxt = trees.commit(*copies, stream=s)
    assert not s.query()  # the calls are still waiting, so the copies that were made above have been made
    del copies, trees, pool, before
    overwrite(*sizes)
    s.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(got, want)
    assert acc.tolist() == [1, 1] and nxt.tolist() == [0, 20]
    w.close()


def test_queries_in_place_of_another_type_or_stride_are_refused():
    w = Setup("8:4x64", "f16", [20], [6], seed=1)
    ld = w.H * w.D
    buf = w.rand(w.N, 2 * ld)
    keep = buf.clone()
    x = dec.dec_tree_qkv(q=buf.data_ptr(), ldq=2 * ld, in_type=dec.DEC_T_F32, q_type=dec.DEC_T_F32, q_out=buf.data_ptr(), ldqo=2 * ld)
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)

    def append(**change):
        y = dec.dec_tree_qkv.from_buffer_copy(x)
        for k, v in change.items():
            setattr(y, k, v)
        return w.trees.L.dec_tree_append(w.trees.handle, 0, C.byref(y), stream)

    assert append(q_type=dec.DEC_T_BF16) == append(ldqo=ld) == append(q_type=dec.DEC_T_F16, ldqo=ld) == dec.DEC_EINVAL
    assert append() == dec.DEC_OK and torch.equal(buf, keep)  # nothing to do to them
    with pytest.raises(dec.DecError):
        w.trees.append(0, buf[:, :ld], None, None, out=buf.view(-1, ld)[: w.N])
    w.close()


@pytest.mark.parametrize("shape, cache", [("16:8x128", "f16"), ("8:4x64", "f32"), ("4:2x32", "f16")])
def test_replays_over_nodes_divided_among_the_sequences_in_other_ways(shape, cache):
    """15 nodes of two sequences: a replay follows any division whose longest tree has the captured one's row tile."""
    w = Setup(shape, cache, [40, 70], [15, 15], seed=3)  # room for either to take all of them
    w.ctx, tables = [40, 70], w.tables
    w.N, w.parents = 15, [random_tree(8, 1), random_tree(7, 2)]
    w.trees.set(w.ctx, w.parents, tables)
    q, k, v = w.rand(15, w.H, w.D), w.rand(15, w.Hkv, w.D), w.rand(15, w.Hkv, w.D)
    qr, out = torch.empty_like(q), torch.empty((15, w.H * w.D), dtype=torch.bfloat16 if cache == "f16" else torch.float32, device="cuda")
    draft = torch.arange(15, dtype=torch.int32, device="cuda")
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (2, 15, 2)]
    rope = RopeTable(w.D, 200)

    def calls():
        w.trees.append(1, q, k, v, rope=rope, out=qr)
        w.trees.attend(1, qr, out=out)
        w.trees.commit(draft, draft, out=outs)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    slab = w.slab.clone()
    for a in (8, 7, 8):  # 16 rows at most: the capture's row tile
        w.parents = [random_tree(a, a), random_tree(15 - a, 20 + a)]
        w.trees.set(w.ctx, w.parents, tables)
        w.slab.copy_(slab)
        out.fill_(float("nan"))
        graph.replay()
        check(w, out, 1, qr)
        got = [x.clone() for x in (qr, w.slab, *outs)]
        w.slab.copy_(slab)
        calls()
        assert all(torch.equal(x, y) for x, y in zip(got, (qr, w.slab, *outs)))
        assert w.trees.status() == 0 and outs[2].tolist() == [0, a]
    for a in (9, 14, 1):  # more rows: attention does nothing and says so, append and commit follow
        w.parents = [random_tree(a, a), random_tree(15 - a, 20 + a)]
        w.trees.set(w.ctx, w.parents, tables)
        out.fill_(7.0)
        graph.replay()
        assert w.trees.status() == dec.DEC_DEV_SHAPE
        assert bool((out == 7.0).all()) and outs[2].tolist() == [0, a]
        want = w.trees.append(1, q, k, v, rope=rope)
        assert torch.equal(qr, want)
    w.trees.set(w.ctx, [8, 7], tables)
    del graph
    w.close()


def test_a_plan_outlives_the_pools_bookkeeping():
    """A closed KvPool keeps its memory: the plan that is set works on, another one is refused."""
    w = Setup("8:4x64", "f16", [20], [6], seed=1)
    q, k = w.rand(w.N, w.H, w.D), w.rand(w.N, w.Hkv, w.D)
    w.trees.append(0, None, k, k)
    want = w.trees.attend(0, q).clone()
    w.pool.close()
    others = [KvPool(w.shape, w.pool.mode, 3) for _ in range(20)]  # host memory of the closed one is used again
    w.trees.append(0, None, k, k)
    assert torch.equal(w.trees.attend(0, q), want)
    with pytest.raises(ValueError):
        w.trees.set(w.ctx, w.parents, w.tables)
    assert torch.equal(w.trees.attend(0, q), want)
    del others
    w.close()
