"""The DEC_DEBUG build over a cache held in 8 bits: a block outside the pool, planted in the device copy of a plan after the
host has validated it, sets DEC_DEV_BOUNDS in every call that reads it there and block 0 takes its place.  The buffer
behind the pool is larger than the pool, so that even a missing check would stay inside it."""

import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import torch
    from decoder_qwen3_step_gb300 import dec
    from decoder_qwen3_step_gb300.trees import DraftTrees, KvPool

    assert dec.LIB_PATH.endswith("libdec_debug.so") and dec.lib().dec_build_flags() & dec.DEC_BUILD_DEBUG
    H, Hkv, D, blocks = 8, 4, 64, 20
    shape = {"vocab": 512, "d_model": 64, "n_layers": 2, "n_heads": H, "n_kv_heads": Hkv, "head_dim": D, "ff_hidden": 64}
    for kind in (dec.DEC_T_I8, dec.DEC_T_E4M3):
        size = 2 * blocks * 2 * Hkv * 16 * D
        buf = torch.randint(0, 0x70, (4 * size,), dtype=torch.uint8).cuda()
        end = size + 2 * blocks * Hkv * 2 * 4  # of the scales
        codes = buf[:size].view(2, blocks, 2, Hkv, 16, D)
        buf[size:].view(torch.float32)[:] = 0.5
        pool = KvPool(shape, dec.DEC_BF16_F16KV, blocks, max_positions=4096, slabs=buf, kv_type=kind)
        pool.alloc(blocks)
        trees = DraftTrees(pool, 2, 64, 8)
        tables, ctx, parents = [[7, 9, 11, 13], [15, 17]], [37, 20], [[-1] * 20, 9]
        ws = trees.workspace
        base = -ws.data_ptr() % 256
        words = ws[base:(ws.numel() - base) // 4 * 4 + base].view(torch.int32)
        g = torch.Generator().manual_seed(1)
        q, k, v = (torch.randn((29, n, D), generator=g).cuda() for n in (H, Hkv, Hkv))
        draft = torch.arange(29, dtype=torch.int32, device="cuda")
        target = torch.full((29,), -1, dtype=torch.int32, device="cuda")
        prior = torch.tensor([18, 20], dtype=torch.int32, device="cuda")  # the walk ends at node 18, and at the second's first
        start = buf.clone()

        def plant(find, at):
            trees.set(ctx, parents, tables)
            n = len(find)
            where = words.unfold(0, n, 1).eq(torch.tensor(find, dtype=torch.int32, device="cuda")).all(1).nonzero()[:, 0]
            assert len(where) == 1, (find, where)
            words[where[0] + at] = blocks + 3 if find[at] < blocks else (blocks + 3) * 16 + find[at] % 16
            buf.copy_(start)

        def clean():
            trees.set(ctx, parents, tables)
            buf.copy_(start)
            out = [trees.append(0, q, k, v).clone(), trees.attend(0, q).clone(), *trees.commit(draft, target, prior), *trees.read(0, layers=2), buf.clone()]
            assert trees.status() == 0
            return out

        want = clean()
        whole = [7, 9, 11, 13, 15, 17]
        plant(whole, 1)
        trees.read(0)
        assert trees.status() == dec.DEC_DEV_BOUNDS
        plant(whole, 1)
        trees.attend(0, q)
        assert trees.status() == dec.DEC_DEV_BOUNDS
        plant([11, 0, 5, 11], 0)  # a page: block, first node, slot, nodes
        trees.append(0, None, k, v)
        assert trees.status() == dec.DEC_DEV_BOUNDS
        assert torch.equal(codes[:, 11], start[:size].view_as(codes)[:, 11]) and not torch.equal(codes[0, 0], start[:size].view_as(codes)[0, 0])
        assert torch.equal(buf[end:], start[end:])
        plant(whole, 2)  # the page that node 18 moves to
        trees.commit(draft, target, prior)
        assert trees.status() == dec.DEC_DEV_BOUNDS
        assert torch.equal(codes[:, 11], start[:size].view_as(codes)[:, 11])
        plant([13 * 16 + 6, 13 * 16 + 7], 0)  # node 17 stays where it is: nobody's slot but its own
        trees.commit(draft, target, prior)
        assert trees.status() == dec.DEC_DEV_BOUNDS
        assert torch.equal(buf[end:], start[end:])
        for x, y in zip(clean(), want):
            assert torch.equal(x, y)
        trees.close()
        pool.close()
    print("8-bit debug build ok")
""")


def test_blocks_outside_the_pool_are_told_and_kept_out():
    from decoder_qwen3_step_gb300 import build

    build.build(debug=True)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env={**os.environ, "DEC_DEBUG": "1"}, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "8-bit debug build ok" in r.stdout, (r.stdout[-3000:], r.stderr[-3000:])
