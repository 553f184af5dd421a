"""Draft trees where calls meet: a wait that has run out and the calls behind
it, streams that order the plan's memory, replays over other trees."""

import ctypes as C

import pytest

torch = pytest.importorskip("torch")

from decoder_qwen3_step_gb300 import dec  # noqa: E402

from .test_gpu_trees import Setup, random_tree  # noqa: E402

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
