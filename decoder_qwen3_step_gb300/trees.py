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
from .inputs import BLOCK_TOKENS
from .runtime import _i32, _ptr, make_config

_empty, _raw_stream = torch.empty, torch._C._cuda_getCurrentRawStream
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
        self.pointer, self.address, self.index = C.pointer(self.rope), self.table.data_ptr(), self.table.get_device()
        with torch.cuda.device(self.table.device):
            dec.check(L.dec_rope_table(C.byref(self.rope), n_positions, C.c_void_p(self.table.data_ptr()), size.value,
                                       C.c_void_p(torch.cuda.current_stream().cuda_stream)), "dec_rope_table")


def tree_batch(ctx, parents, tables):
    """A dec_tree_batch from lists per sequence: cached tokens, parents of the
    nodes (an int n stands for a chain of n), pool blocks.  Returns the struct
    and the arrays that it points to."""
    nodes = [np.arange(-1, int(p) - 1, dtype=np.int32) if np.ndim(p) == 0 else np.asarray(p, dtype=np.int32) for p in parents]
    if not len(ctx) == len(nodes) == len(tables):
        raise ValueError("one context, one tree and one table per sequence")
    start = _i32(np.concatenate([[0], np.cumsum([len(p) for p in nodes])]) if nodes else [0])
    width = max([len(t) for t in tables] + [1])
    tab = np.zeros((max(len(tables), 1), width), dtype=np.int32)
    for i, t in enumerate(tables):
        tab[i, :len(t)] = t
        if len(t) < width and len(t) * BLOCK_TOKENS < ctx[i] + len(nodes[i]):
            tab[i, len(t):] = -1  # the library refuses the table: a filled-up one would name somebody's block
    flat = np.concatenate(nodes + [np.zeros(1, dtype=np.int32)])  # never empty
    arrays = (start, _i32(ctx if len(ctx) else [0]), flat, tab)
    return dec.dec_tree_batch(len(nodes), int(start[-1]), *(_ptr(a) for a in arrays), width), arrays


def _used_on(stream, *tensors):
    """Tensors that a call on a given stream reads or writes: their memory is not reused before it has."""
    for x in tensors:
        if x is not None:
            x.record_stream(stream)


class DraftTrees:
    """The plan of a step's draft trees over one pool (a KvPool or a Decoder).

    Calls run on the current stream, or on `stream`.  Either way the caller
    orders them behind the work that fills their inputs; the tensors given to
    a call with `stream` may be dropped right after it.  What a captured graph
    uses (this plan, its pool, the tensors of the calls) has to be kept for as
    long as the graph is replayed."""

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
        self._streams = set()  # that calls were made on
        self._heads, self._kv_heads, self._dim = self.cfg.n_heads, self.cfg.n_kv_heads, self.cfg.head_dim
        # a step makes these calls for every layer: the lookups are done once
        self._append, self._attend, self._commit = self.L.dec_tree_append, self.L.dec_tree_attend, self.L.dec_tree_commit
        self._qkv = dec.dec_tree_qkv()
        self._out_type = torch.float32 if self.cfg.mode == dec.DEC_FP32 else torch.bfloat16

    def _stream(self, stream):
        raw = stream.cuda_stream if stream is not None else _raw_stream(self._index)
        if raw not in self._streams:  # the plan's memory and the pool's must not be given away while this stream reads them
            s = stream if stream is not None else torch.cuda.current_stream(self._index)
            for x in (self.workspace, self.pool.slabs):
                x.record_stream(s)
            self._streams.add(raw)
        return raw

    def _new(self, shape, dtype, stream):
        """An output that lives on the stream its kernel runs on."""
        if stream is None:
            return _empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return _empty(shape, dtype=dtype, device=self.device)

    def _rows(self, x, name, heads):
        """Row stride and type of a [nodes, heads, head_dim] (or [nodes, heads * head_dim]) tensor."""
        st, shape, dim = x.stride(), x.shape, self._dim
        good = (shape == (self.n_tokens, heads, dim) and st[2] == 1 and (st[1] == dim or heads == 1)) or (
            shape == (self.n_tokens, heads * dim) and st[1] == 1)
        if not good or x.dtype not in _TYPES or x.get_device() != self._index:
            raise ValueError(f"{name}: need a [{self.n_tokens}, {heads}, {dim}] tensor of f32, f16 or bf16 on cuda:{self._index}"
                             f" with rows of back-to-back heads, got {x.dtype} {tuple(shape)} strides {st} on {x.device}")
        return x.data_ptr(), (st[0] if self.n_tokens > 1 else heads * dim), _TYPES[x.dtype]

    def set(self, ctx, parents, tables, stream=None) -> None:
        """This step's trees: cached tokens, parents (an int n: a chain of n) and block table of every sequence."""
        if not self.pool.pool:
            raise ValueError("the pool is closed")
        b, keep = tree_batch(ctx, parents, tables)
        dec.check(self.L.dec_tree_set(self.handle, C.byref(b), self._stream(stream)), "dec_tree_set")
        self.n_seqs, self.n_tokens = b.n_seqs, b.n_tokens

    def append(self, layer: int, q, k, v, rope: RopeTable | None = None, q_norm=None, k_norm=None, q_type=torch.float32,
               out=None, stream=None):
        """Norm (where gains are given), rotate, and write keys and values to
        the nodes' slots; returns the queries [nodes, heads, head_dim].  q, or k and v, may be None."""
        x, kind = self._qkv, None  # the struct is read during the call only; every field below is set each time
        if q is not None:
            x.q, x.ldq, kind = self._rows(q, "q", self._heads)
        else:
            x.q = x.q_out = None
        if k is not None:
            x.k, x.ldk, kind_k = self._rows(k, "k", self._kv_heads)
            if kind is not None and kind != kind_k:
                raise ValueError("q, k and v must have one type")
            kind = kind_k
        else:
            x.k = None
        if v is not None:
            x.v, x.ldv, kind_v = self._rows(v, "v", self._kv_heads)
            if kind is not None and kind != kind_v:
                raise ValueError("q, k and v must have one type")
            kind = kind_v
        else:
            x.v = None
        x.in_type = kind or 0
        x.q_norm = self._gain(q_norm, "q_norm")
        x.k_norm = self._gain(k_norm, "k_norm")
        if rope is not None:
            if rope.index != self._index:
                raise ValueError(f"the rotary table is not on cuda:{self._index}")
            x.rope, x.rope_table, x.rope_positions = rope.pointer, rope.address, rope.n_positions
        else:
            x.rope = None
        # outputs last: an allocation close behind the call before waits for that call's doorbell
        if out is not None:
            x.q_out, x.ldqo, x.q_type = self._rows(out, "out", self._heads)
        elif q is not None:
            out = self._new((self.n_tokens, self._heads, self._dim), q_type, stream)
            x.q_out, x.ldqo, x.q_type = out.data_ptr(), self._heads * self._dim, _TYPES[q_type]
        if stream is not None:
            _used_on(stream, q, k, v, q_norm, k_norm, out, rope and rope.table)
        code = self._append(self.handle, layer, x, self._stream(stream))
        if code:
            dec.check(code, "dec_tree_append")
        return out

    def _gain(self, g, name):
        if g is None:
            return None
        if g.dtype is not torch.float32 or g.shape != (self._dim,) or not g.is_contiguous() or g.get_device() != self._index:
            raise ValueError(f"{name}: need [{self._dim}] f32 on cuda:{self._index}")
        return g.data_ptr()

    def attend(self, layer: int, q, out=None, out_type=None, stream=None):
        """Attention of every node over what it sees: [nodes, heads * head_dim]
        (default type: f32 for an fp32 cache, else bf16)."""
        p, ld, kind = self._rows(q, "q", self._heads)
        if out is None:
            out_type = out_type or self._out_type
            out = self._new((self.n_tokens, self._heads * self._dim), out_type, stream)
            po, ldo, kind_o = out.data_ptr(), self._heads * self._dim, _TYPES[out_type]
        else:
            po, ldo, kind_o = self._rows(out, "out", self._heads)
        if stream is not None:
            _used_on(stream, q, out)
        code = self._attend(self.handle, layer, p, kind, ld, po, kind_o, ldo, self._stream(stream))
        if code:
            dec.check(code, "dec_tree_attend")
        return out

    def _ids(self, t, name, n):
        if t.dtype is not torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name}: need [{n}] int32 on cuda:{self._index}")
        return t.data_ptr()

    def commit(self, draft, target, prior=None, out=None, stream=None):
        """Accept along the chosen tokens and compact the cache: device int32
        (accepted [sequences], path [nodes], next [sequences])."""
        n, s = self.n_tokens, self.n_seqs
        ids = self._ids(draft, "draft", n), self._ids(target, "target", n), None if prior is None else self._ids(prior, "prior", s)
        if out is None:  # three tensors: one buffer and its views cost twice as much host time
            out = tuple(self._new(x, torch.int32, stream) for x in (s, n, s))
            a, p, x = out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr()
        else:
            a, p, x = self._ids(out[0], "accepted", s), self._ids(out[1], "path", n), self._ids(out[2], "next", s)
        if stream is not None:
            _used_on(stream, draft, target, prior, *out)
        code = self._commit(self.handle, *ids, a, p, x, self._stream(stream))
        if code:
            dec.check(code, "dec_tree_commit")
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
