"""Draft trees at the ends of what attention's weights hold: scores of any size, pages of an 8-bit cache whose scales lie
some powers of two apart."""

import math

import pytest

torch = pytest.importorskip("torch")

from tests.q8_reference import KINDS, codes_of  # noqa: E402
from tests.test_gpu_q8 import Setup8  # noqa: E402
from tests.test_gpu_trees import Setup  # noqa: E402

pytestmark = pytest.mark.gpu


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
