// tree_common.cuh - device helpers shared by the draft-tree attention kernels.
#pragma once

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

// One unit of attention work: the rows row0 .. row0+rows-1 (row r: node r / G,
// query head r % G of the group) of one sequence and KV head.
struct TreeUnit {
  int seq, head, row_tile, n_row_tiles;
  int node0, ctx, nodes;  // the sequence's first node, cached tokens, nodes
  int tiles;              // key tiles of ctx + nodes keys
};

__device__ __forceinline__ void tree_unit_load(const TreeMeta& m, int G, int R, TreeUnit& u) {
  u.node0 = __ldg(m.seq_start + u.seq);
  u.nodes = __ldg(m.seq_start + u.seq + 1) - u.node0;
  u.ctx = __ldg(m.ctx + u.seq);
  u.tiles = (u.ctx + u.nodes + m.tile_keys - 1) / m.tile_keys;
  u.n_row_tiles = (u.nodes * G + R - 1) / R;
}
// The unit after u (sequences without nodes have none).
__device__ __forceinline__ void tree_unit_next(const TreeMeta& m, int G, int R, int Hkv, TreeUnit& u) {
  if (++u.row_tile < u.n_row_tiles) return;
  u.row_tile = 0;
  if (++u.head < Hkv) return;
  u.head = 0;
  do {
    ++u.seq;
  } while (u.seq < m.S && __ldg(m.seq_start + u.seq + 1) == __ldg(m.seq_start + u.seq));
  if (u.seq < m.S) tree_unit_load(m, G, R, u);
}

// Whether node `node` (numbered over the batch) sees node j of its sequence.
__device__ __forceinline__ bool tree_sees(const TreeMeta& m, int node, int j) {
  return (__ldg(m.anc + (size_t)node * m.words + (j >> 5)) >> (j & 31)) & 1u;
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

// Slot of a CTA's record: its first unit when that began in an earlier CTA, or
// the one it leaves unfinished.
__device__ __forceinline__ float* tree_record(const TreeAttendArgs& a, int cta, bool leaves) {
  return a.part + ((size_t)cta * 2 + leaves) * a.m.row_tile * (a.d.D + 2);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Load the queries of a unit's row tile as f16 into shared memory: warp w of
// W takes rows w, w + W, ..., eight in flight (a row's load takes about a
// microsecond from HBM; one at a time, 128 rows cost more than a dozen key
// tiles).  Each row is scaled by a power of two so that its largest magnitude
// lies in [1, 2): f16 then rounds every channel by at most 2^-12 of that,
// whatever the queries' range; fac[r] takes the row's score factor.  put(r,
// lane, halves 4 lane .. 4 lane + 3).  Rows past the last are zeros.
template <int D, int R, int W, typename F>
__device__ __forceinline__ void tree_load_queries(const TreeAttendArgs& a, const TreeUnit& u, int G, int w, float* fac, F&& put) {
  constexpr int kU = R / W < 8 ? R / W : 8;
  const int lane = threadIdx.x & 31, rows = min(R, u.nodes * G - u.row_tile * R);
  for (int r0 = w; r0 < R; r0 += W * kU) {
    float4 v[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int r = r0 + i * W, row = u.row_tile * R + r;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows && lane * 4 < D)
        v[i] = tree_load4(a.q, a.q_type, (u.node0 + row / G) * a.ldq + (int64_t)(u.head * G + row % G) * D + lane * 4);
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int r = r0 + i * W;
      const float mx = warp_max(fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
      // the factor 2^-e, 2^e <= mx < 2^(e+1); rows of zeros, subnormals or infinities stay as they are
      const int e = (int)(__float_as_uint(mx) >> 23);
      const bool scaled = e > 0 && e < 255;
      const float f = scaled ? __uint_as_float((uint32_t)max(254 - e, 1) << 23) : 1.f;
      const __half2 lo = __floats2half2_rn(v[i].x * f, v[i].y * f), hi = __floats2half2_rn(v[i].z * f, v[i].w * f);
      if (lane * 4 < D) put(r, lane, make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi)));
      if (lane == 0) fac[r] = a.scale_log2 * (scaled ? 1.f / f : 1.f);
    }
  }
}

}  // namespace dec
