"""Draft trees over the paged KV cache: device buffers through torch, every
operation in libdec (``dec_tree_*`` and ``dec_rope_table`` in include/dec.h).

A verification step of a program that runs its own projections::

    pool = KvPool(shape, dec.DEC_BF16_F16KV, n_blocks)        # or a Decoder
    rope = RopeTable(rot_dim=128, n_positions=4096)
    trees = DraftTrees(pool, max_seqs=32, max_tokens=2048, max_blocks=256)
    trees.set(ctx, parents, tables)                            # once a step
    for layer in range(n_layers):
        q = trees.append(layer, q_raw, k_raw, v_raw, rope=rope, q_norm=gq, k_norm=gk)
        o = trees.attend(layer, q)
    accepted, path, after = trees.commit(draft_ids, chosen_ids)
"""

from __future__ import annotations

import ctypes as C

import numpy as np
import torch

from . import dec
from .runtime import _i32, _ptr, make_config

_TYPES = {torch.float32: dec.DEC_T_F32, torch.float16: dec.DEC_T_F16, torch.bfloat16: dec.DEC_T_BF16}


class KvPool:
    """A paged KV pool without a model: the slab buffer (allocated here, or
    the caller's) and libdec's block bookkeeping."""

    def __init__(self, shape: dict, mode: int, n_blocks: int, max_positions: int = 4096, device: str = "cuda:0",
                 slabs: torch.Tensor | None = None):
        self.L = dec.lib()
        self.shape, self.mode, self.n_blocks = dict(shape), mode, n_blocks
        self.cfg = make_config(shape, mode, max_positions)
        size = C.c_size_t()
        dec.check(self.L.dec_pool_bytes(C.byref(self.cfg), n_blocks, C.byref(size)), "dec_pool_bytes")
        if slabs is None:
            slabs = torch.zeros(size.value, dtype=torch.uint8, device=device)
        assert slabs.is_cuda and slabs.is_contiguous()
        self.slabs, self.device = slabs, slabs.device
        h = C.c_void_p()
        dec.check(self.L.dec_pool_create(C.byref(self.cfg), n_blocks, C.c_void_p(slabs.data_ptr()),
                                         slabs.numel() * slabs.element_size(), C.byref(h)), "dec_pool_create")
        self.pool = h

    def alloc(self, n: int) -> list:
        ids = (C.c_int32 * max(n, 1))()
        dec.check(self.L.dec_pool_alloc(self.pool, n, ids), "dec_pool_alloc")
        return list(ids[:n])

    def release(self, ids) -> None:
        for i in ids:
            dec.check(self.L.dec_pool_release(self.pool, int(i)), "dec_pool_release")

    def close(self):
        if getattr(self, "pool", None):
            self.L.dec_pool_destroy(self.pool)
            self.pool = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class RopeTable:
    """A rotary table (dec_rope): positions 0 .. n_positions - 1 of the first
    rot_dim channels of a head."""

    def __init__(self, rot_dim: int, n_positions: int, base: float = 1e6, layout: int = dec.DEC_ROPE_HALF,
                 scaling: int = dec.DEC_ROPE_PLAIN, factor: float = 1.0, orig_positions: int = 0, low: float = 0.0,
                 high: float = 0.0, attn_factor: float = 1.0, device: str = "cuda:0"):
        L = dec.lib()
        self.rope = dec.dec_rope(rot_dim, layout, scaling, orig_positions, base, factor, low, high, attn_factor)
        self.n_positions = n_positions
        size = C.c_size_t()
        dec.check(L.dec_rope_table_bytes(C.byref(self.rope), n_positions, C.byref(size)), "dec_rope_table_bytes")
        self.table = torch.empty((n_positions, rot_dim // 2, 2), dtype=torch.float32, device=device)
        with torch.cuda.device(self.table.device):
            dec.check(L.dec_rope_table(C.byref(self.rope), n_positions, C.c_void_p(self.table.data_ptr()), size.value,
                                       C.c_void_p(torch.cuda.current_stream().cuda_stream)), "dec_rope_table")


def tree_batch(ctx, parents, tables):
    """A dec_tree_batch from lists per sequence: cached tokens, parents of the
    nodes (an int n stands for a chain of n), pool blocks.  Returns the struct
    and the arrays that it points to."""
    nodes = [list(range(-1, p - 1)) if isinstance(p, int) else list(p) for p in parents]
    if not len(ctx) == len(nodes) == len(tables):
        raise ValueError("one context, one tree and one table per sequence")
    start = _i32(np.concatenate([[0], np.cumsum([len(p) for p in nodes])]) if nodes else [0])
    width = max([len(t) for t in tables] + [1])
    tab = np.zeros((max(len(tables), 1), width), dtype=np.int32)
    for i, t in enumerate(tables):
        tab[i, :len(t)] = t
    flat = _i32([p for tree in nodes for p in tree] or [0])
    arrays = (start, _i32(ctx if len(ctx) else [0]), flat, tab)
    return dec.dec_tree_batch(len(nodes), int(start[-1]), *(_ptr(a) for a in arrays), width), arrays


class DraftTrees:
    """The plan of a step's draft trees over one pool (a KvPool or a Decoder)."""

    def __init__(self, pool, max_seqs: int, max_tokens: int, max_blocks: int):
        self.L = dec.lib()
        self.pool, self.cfg, self.device = pool, pool.cfg, pool.device
        self._index = self.device.index if self.device.index is not None else torch.cuda.current_device()
        size = C.c_size_t()
        with torch.cuda.device(self._index):
            dec.check(self.L.dec_tree_workspace_bytes(pool.pool, max_seqs, max_tokens, max_blocks, C.byref(size)),
                      "dec_tree_workspace_bytes")
            self.workspace = torch.empty(size.value + 256, dtype=torch.uint8, device=self.device)
            base = (self.workspace.data_ptr() + 255) & ~255
            h = C.c_void_p()
            dec.check(self.L.dec_tree_create(pool.pool, max_seqs, max_tokens, max_blocks, C.c_void_p(base), size.value,
                                             C.byref(h)), "dec_tree_create")
        self.handle = h
        self.n_tokens = self.n_seqs = 0
        self._width = {"q": (self.cfg.n_heads, self.cfg.head_dim), "k": (self.cfg.n_kv_heads, self.cfg.head_dim),
                       "v": (self.cfg.n_kv_heads, self.cfg.head_dim)}
        self._out_type = torch.float32 if self.cfg.mode == dec.DEC_FP32 else torch.bfloat16

    def _stream(self, stream):
        return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self._index)

    def _new(self, shape, dtype, stream):
        """An output that lives on the stream its kernel runs on."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _rows(self, x, name, what="q"):
        """Row stride and type of a [nodes, heads, head_dim] (or [nodes, heads * head_dim]) tensor."""
        heads, dim = self._width[what]
        st, dt = x.stride(), _TYPES.get(x.dtype)
        good = (x.shape == (self.n_tokens, heads, dim) and st[2] == 1 and (st[1] == dim or heads == 1)) or (
            x.shape == (self.n_tokens, heads * dim) and st[1] == 1)
        if dt is None or not good or x.get_device() != self._index:
            raise ValueError(f"{name}: need a [{self.n_tokens}, {heads}, {dim}] tensor of f32, f16 or bf16 on cuda:{self._index}"
                             f" with rows of back-to-back heads, got {x.dtype} {tuple(x.shape)} strides {st} on {x.device}")
        return x.data_ptr(), (st[0] if self.n_tokens > 1 else heads * dim), dt

    def set(self, ctx, parents, tables, stream=None) -> None:
        """This step's trees: cached tokens, parents (an int n: a chain of n) and block table of every sequence."""
        b, keep = tree_batch(ctx, parents, tables)
        dec.check(self.L.dec_tree_set(self.handle, C.byref(b), self._stream(stream)), "dec_tree_set")
        self.n_seqs, self.n_tokens = b.n_seqs, b.n_tokens

    def append(self, layer: int, q, k, v, rope: RopeTable | None = None, q_norm=None, k_norm=None, q_type=torch.float32,
               out=None, stream=None):
        """Norm (where gains are given), rotate, and write keys and values to
        the nodes' slots; returns the queries [nodes, heads, head_dim].  q, or k and v, may be None."""
        x = dec.dec_tree_qkv()
        kinds = set()
        for name, t in (("q", q), ("k", k), ("v", v)):
            if t is not None:
                p, ld, kind = self._rows(t, name, name)
                setattr(x, name, p)
                setattr(x, "ld" + name, ld)
                kinds.add(kind)
        if len(kinds) > 1:
            raise ValueError("q, k and v must have one type")
        x.in_type = kinds.pop() if kinds else 0
        for name, g in (("q_norm", q_norm), ("k_norm", k_norm)):
            if g is not None:
                if g.dtype != torch.float32 or g.shape != (self.cfg.head_dim,) or not g.is_contiguous() or g.get_device() != self._index:
                    raise ValueError(f"{name}: need [{self.cfg.head_dim}] f32 on cuda:{self._index}")
                setattr(x, name, g.data_ptr())
        if rope is not None:
            if rope.table.get_device() != self._index:
                raise ValueError(f"the rotary table is not on cuda:{self._index}")
            x.rope, x.rope_table, x.rope_positions = C.pointer(rope.rope), rope.table.data_ptr(), rope.n_positions
        if q is not None:
            if out is None:
                out = self._new((self.n_tokens, *self._width["q"]), q_type, stream)
            x.q_out, x.ldqo, x.q_type = self._rows(out, "out")
        dec.check(self.L.dec_tree_append(self.handle, layer, x, self._stream(stream)), "dec_tree_append")
        return out

    def attend(self, layer: int, q, out=None, out_type=None, stream=None):
        """Attention of every node over what it sees: [nodes, heads * head_dim]
        (default type: f32 for an fp32 cache, else bf16)."""
        p, ld, kind = self._rows(q, "q")
        if out is None:
            out = self._new((self.n_tokens, self.cfg.n_heads * self.cfg.head_dim), out_type or self._out_type, stream)
        po, ldo, kind_o = self._rows(out, "out")
        dec.check(self.L.dec_tree_attend(self.handle, layer, p, kind, ld, po, kind_o, ldo, self._stream(stream)),
                  "dec_tree_attend")
        return out

    def commit(self, draft, target, prior=None, out=None, stream=None):
        """Accept along the chosen tokens and compact the cache: device int32
        (accepted [sequences], path [nodes], next [sequences])."""
        want = [("draft", draft, self.n_tokens), ("target", target, self.n_tokens), ("prior", prior, self.n_seqs)]
        if out is None:
            buf = self._new((self.n_tokens + 2 * self.n_seqs,), torch.int32, stream)
            out = buf.split([self.n_seqs, self.n_tokens, self.n_seqs])
        want += [("accepted", out[0], self.n_seqs), ("path", out[1], self.n_tokens), ("next", out[2], self.n_seqs)]
        for name, t, n in want:
            if t is not None and (t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != self._index):
                raise ValueError(f"{name}: need [{n}] int32 on cuda:{self._index}")
        dec.check(self.L.dec_tree_commit(self.handle, draft.data_ptr(), target.data_ptr(),
                                         prior.data_ptr() if prior is not None else None, out[0].data_ptr(),
                                         out[1].data_ptr(), out[2].data_ptr(), self._stream(stream)), "dec_tree_commit")
        return out

    def status(self, stream=None) -> int:
        f = C.c_uint32()
        dec.check(self.L.dec_tree_status(self.handle, self._stream(stream), C.byref(f)), "dec_tree_status")
        return f.value

    def close(self):
        if getattr(self, "handle", None):
            self.L.dec_tree_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
