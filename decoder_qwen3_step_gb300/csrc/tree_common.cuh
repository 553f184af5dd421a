// tree_common.cuh - device helpers shared by the draft-tree attention kernels.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "tree.h"

namespace dec {

// Whether the launch fits the plan that is on the device now: a captured call
// replayed after dec_tree_set gave the plan another shape does nothing but
// raise kErrShape.  The row tile only matters to the attention kernels.
__device__ __forceinline__ bool tree_shape_ok(const TreeMeta& m, bool rows = false) {
  const int4 h = *reinterpret_cast<const int4*>(m.hdr);
  const bool ok = h.x == m.S && h.y == m.N && h.z == m.words && (!rows || h.w == m.row_tile);
  if (!ok && threadIdx.x == 0) atomicOr(m.err, kErrShape);
  return ok;
}

// One unit of attention work: the rows row_tile * R .. of one sequence and KV
// head (row r: node r >> gs, query head r & (2^gs - 1) of the group).
struct TreeUnit {
  int q, head, row_tile, step;
  int node0, nodes, ctx, tab;
  int tiles;  // key tiles of ctx + nodes keys
};
__device__ __forceinline__ void tree_unit_seq(const TreeMeta& m, const int4& s, TreeUnit& u) {
  u.node0 = s.x;
  u.nodes = s.y;
  u.ctx = s.z;
  u.tab = s.w;
  u.tiles = (u.ctx + u.nodes + m.tile_keys - 1) / m.tile_keys;
}
// The unit a CTA starts with.
__device__ __forceinline__ TreeUnit tree_unit_first(const TreeMeta& m, const TreeCut& c) {
  TreeUnit u{c.q, c.head, c.row_tile, max(c.step, 1), 0, 0, 0, 0, 0};
  tree_unit_seq(m, make_int4(c.s.node0, c.s.nodes, c.s.ctx, c.s.tab), u);
  return u;
}
// The unit after u; there must be one.
__device__ __forceinline__ void tree_unit_next(const TreeMeta& m, int gs, int R, int Hkv, TreeUnit& u) {
  u.row_tile += u.step;
  if (u.row_tile * R < u.nodes << gs) return;
  u.row_tile %= u.step;
  if (++u.head < Hkv) return;
  u.head = 0;
  ++u.q;
  tree_unit_seq(m, __ldg(reinterpret_cast<const int4*>(m.seqs + u.q)), u);
}

// Pool block blk, as the plan names it.  DEC_DEBUG builds: block 0 in place of one outside the pool, and kErrBounds.
__device__ __forceinline__ int tree_block(const TreeMeta& m, int n_blocks, int blk) {
#ifdef DEC_DEBUG
  if ((unsigned)blk >= (unsigned)n_blocks) {
    atomicOr(m.err, kErrBounds);
    return 0;
  }
#else
  (void)m;
  (void)n_blocks;
#endif
  return blk;
}

// Whether node `node` (numbered over the batch) sees node j of its sequence.
__device__ __forceinline__ bool tree_sees(const TreeMeta& m, int node, int j) {
  return (__ldg(m.anc + (size_t)node * m.words + (j >> 5)) >> (j & 31)) & 1u;
}

// Whether any of eight halves is infinite or NaN (its exponent bits, all ones, carry into the sign's place), and a pair of
// halves with those set to 0.
__device__ __forceinline__ uint32_t tree_not_finite(uint4 x) {
  return (((x.x & 0x7C007C00u) + 0x04000400u) | ((x.y & 0x7C007C00u) + 0x04000400u) | ((x.z & 0x7C007C00u) + 0x04000400u) |
          ((x.w & 0x7C007C00u) + 0x04000400u)) & 0x80008000u;
}
__device__ __forceinline__ uint32_t tree_finite_or_0(uint32_t w) {
  return w & ~(((w & 0x7C00u) == 0x7C00u ? 0xFFFFu : 0u) | ((w & 0x7C000000u) == 0x7C000000u ? 0xFFFF0000u : 0u));
}

// Which of the nodes j .. j + 31 of its sequence a row of the mask (m.words words) sees, bit 0 node j; j > -32, and
// negative numbers are cached tokens, which every row sees.  Two loads without a branch: a branch and a load per key cost
// the tile that holds the nodes 2 us of serial latency.
__device__ __forceinline__ uint32_t tree_window(const TreeMeta& m, const uint32_t* row, int j) {
  const int w = j >> 5;
  const uint32_t a = __ldg(row + min(max(w, 0), m.words - 1)), b = __ldg(row + min(w + 1, m.words - 1));
  return __funnelshift_r(w < 0 ? 0xffffffffu : w < m.words ? a : 0u, w + 1 < m.words ? b : 0u, j & 31);
}

// The two 16-bit elements of a word as fp32 (both conversions are exact).
template <typename T>
__device__ __forceinline__ float2 tree_pair(uint32_t w);
template <>
__device__ __forceinline__ float2 tree_pair<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 tree_pair<bf16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ float tree_load(const void* p, int type, int64_t i) {
  if (type == kTreeF32) return reinterpret_cast<const float*>(p)[i];
  if (type == kTreeF16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  return __bfloat162float(reinterpret_cast<const bf16*>(p)[i]);
}
__device__ __forceinline__ void tree_store(void* p, int type, int64_t i, float v) {
  if (type == kTreeF32) reinterpret_cast<float*>(p)[i] = v;
  else if (type == kTreeF16) reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
  else reinterpret_cast<bf16*>(p)[i] = __float2bfloat16_rn(v);
}
// Four consecutive elements (the first a multiple of 4) as fp32.
__device__ __forceinline__ float4 tree_load4(const void* p, int type, int64_t i) {
  if (type == kTreeF32) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
  if (type == kTreeF16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 tree_load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <typename T>
__device__ __forceinline__ float4 tree_load4(const T* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 x = tree_pair<T>(u.x), y = tree_pair<T>(u.y);
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ void tree_store4(void* p, int type, int64_t i, float4 v) {
  if (type == kTreeF32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = v;
    return;
  }
  uint2 u;
  if (type == kTreeF16) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) = u;
}

// ---- the walk of a commit ---------------------------------------------------------
// From the root of sequence s (taken as certain, or as prior chose) down to the child whose token is the one the model
// chose at its parent, the lowest such node, until there is none.  The nodes are b .. b + T - 1; a block of kThreads threads
// fills path[] (shared, as child[] and n_path) and returns its length, 0 where the plan does not fit the launch (!ok); `tell`:
// this block writes the call's outputs.  Waits for the kernels before.
template <int kThreads>
__device__ __forceinline__ int tree_walk(const TreeCommitArgs& a, int s, int b, int T, bool ok, bool tell, int* child, int* path, int* n_path) {
  for (int i = threadIdx.x; i <= T; i += kThreads) child[i] = INT_MAX;
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return 0;
  __syncthreads();
  for (int i = threadIdx.x; i < T; i += kThreads) {
    const int p = __ldg(a.m.parents + b + i);
    if (p < -1) continue;  // padding
    const bool good = p >= 0 ? a.draft[b + i] == a.target[b + p] : !a.prior || a.draft[b + i] == a.prior[s];
    if (good) atomicMin(&child[p + 1], i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    for (int at = child[0]; at != INT_MAX; at = child[at + 1]) path[n++] = at;
    *n_path = n;
  }
  __syncthreads();
  const int n = *n_path;
  if (tell) {
    for (int i = threadIdx.x; i < T; i += kThreads) a.path[b + i] = i < n ? path[i] : -1;
    if (threadIdx.x == 0) {
      a.accepted[s] = n;
      a.next[s] = n ? a.target[b + path[n - 1]] : a.prior ? a.prior[s] : -1;
    }
  }
  return n;
}

// Slot of a CTA's record: its first unit when that began in an earlier CTA, or
// the one it leaves unfinished.
__device__ __forceinline__ float* tree_record(const TreeAttendArgs& a, int cta, bool leaves) {
  return a.part + ((size_t)cta * 2 + leaves) * a.m.row_tile * (a.d.D + 2);
}

// ---- joining shared units without a second launch -------------------------------
// The CTA that starts a unit (and whose run ends in it) joins the parts of the
// CTAs that finish it: each of those publishes its record, the first thing of
// its run, by adding 1 to its flag (from a warp that has nothing else to do: the
// fence took the softmax warps up to 3 us), and the joining CTA waits for the
// flags at its own end and subtracts the 1 at its exit.  Both happen in every
// call, in whichever order once a wait has run out, so a flag is 0 again when
// the call has ended and a part that came too late is never taken for the next
// call's.  What a CTA waits for lies behind its place, and the last place is
// the first block's, so it waits only for blocks that were started before it (a
// place from an atomic ticket instead cost 3 us of a 9 us call).
__device__ __forceinline__ int tree_place() { return gridDim.x - 1 - blockIdx.x; }
// After a barrier behind the record's stores; one thread.
__device__ __forceinline__ void tree_publish(const TreeMeta& m, int place) {
  __threadfence();
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(m.flags + place), "r"(1u) : "memory");
}
// Wait for the record of `place` (one thread; a barrier then spreads it).  Gives up after limit_ns.
__device__ __forceinline__ void tree_await(const TreeMeta& m, int place, uint64_t limit_ns = 1000000000ull) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(m.flags + place) : "memory");
    if (v == 1u) break;
    uint64_t now;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
    if (!t0) t0 = now;
    if (now - t0 > limit_ns) {
      atomicOr(m.err, kErrTimeout);
      break;
    }
  }
  __threadfence();
}
// The joining CTA is done with the record of `place`; one thread, after every wait for it.
__device__ __forceinline__ void tree_retire(const TreeMeta& m, int place) { atomicSub(m.flags + place, 1u); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Load R rows of a unit's queries, from row0 on (at least one of them is
// there), as f16 into shared memory.  D/8 lanes
// share a row (eight channels each), so a warp reads 32/(D/8) rows at a time
// and has up to kMaxU such groups in flight; W warps split the rows.  The code has no
// branch and no division per row: a first version with both, one row per warp
// and step, took 0.7 us a row on instruction latency alone.
// Each row is scaled by a power of two so that its largest magnitude lies in
// [1, 2): f16 then rounds every channel by at most 2^-11 of that, whatever the
// queries' range; fac[r] takes the row's score factor.  put(r, channel / 8,
// eight halves).  Rows past the last are zeros.
template <int D, int R, int W, int kMaxU, typename T, typename F>
__device__ __forceinline__ void tree_load_queries_of(const TreeAttendArgs& a, const TreeUnit& u, int row0, int w, float* fac, F&& put) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kSteps = R / (W * kRows), kU = kSteps < kMaxU ? kSteps : kMaxU;
  constexpr bool kWide = sizeof(T) == 4;
  static_assert(kSteps >= 1 && kSteps % kU == 0, "rows split evenly");
  const int lane = threadIdx.x & 31, x = lane % kLanes, gs = a.d.gs;
  const int rows = min(R, (u.nodes << gs) - row0);
  const T* q = reinterpret_cast<const T*>(a.q) + (int64_t)u.node0 * a.ldq + (u.head << gs) * D + x * 8;
#pragma unroll 1
  for (int s = 0; s < kSteps; s += kU) {
    uint4 raw[kU][kWide ? 2 : 1];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int row = row0 + min(((s + i) * W + w) * kRows + lane / kLanes, rows - 1);
      const T* p = q + (int64_t)(row >> gs) * a.ldq + (row & ((1 << gs) - 1)) * D;
      if constexpr (kWide) {
        raw[i][0] = *reinterpret_cast<const uint4*>(p);
        raw[i][1] = *reinterpret_cast<const uint4*>(p + 4);
      } else {  // rows are aligned to four elements: 8 bytes
        const uint2 a0 = *reinterpret_cast<const uint2*>(p), a1 = *reinterpret_cast<const uint2*>(p + 4);
        raw[i][0] = make_uint4(a0.x, a0.y, a1.x, a1.y);
      }
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int r = ((s + i) * W + w) * kRows + lane / kLanes;
      float v[8];
      if constexpr (kWide) {
        const uint32_t b[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w, raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(b[e]);
      } else {
        const uint32_t b[4] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = tree_pair<T>(b[e]);
          v[2 * e] = f.x;
          v[2 * e + 1] = f.y;
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // the factor 2^-e, 2^e <= mx < 2^(e+1); rows of zeros, subnormals or infinities stay as they are
      const int e = (int)(__float_as_uint(mx) >> 23);
      const bool scaled = e > 0 && e < 255;
      const int fe = max(254 - e, 1);  // its exponent bits; the inverse has 254 - fe
      const float f = r >= rows ? 0.f : scaled ? __uint_as_float((uint32_t)fe << 23) : 1.f;
      uint32_t h[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const __half2 y = __floats2half2_rn(v[2 * z] * f, v[2 * z + 1] * f);
        h[z] = r >= rows ? 0u : *reinterpret_cast<const uint32_t*>(&y);
      }
      put(r, x, make_uint4(h[0], h[1], h[2], h[3]));
      if (x == 0) fac[r] = a.scale_log2 * (scaled ? __uint_as_float((uint32_t)max(254 - fe, 1) << 23) : 1.f);
    }
  }
}
template <int D, int R, int W, int kMaxU, typename F>
__device__ __forceinline__ void tree_load_queries(const TreeAttendArgs& a, const TreeUnit& u, int row0, int w, float* fac, F&& put) {
  if (a.q_type == kTreeF32) tree_load_queries_of<D, R, W, kMaxU, float>(a, u, row0, w, fac, put);
  else if (a.q_type == kTreeF16) tree_load_queries_of<D, R, W, kMaxU, __half>(a, u, row0, w, fac, put);
  else tree_load_queries_of<D, R, W, kMaxU, bf16>(a, u, row0, w, fac, put);
}

}  // namespace dec
