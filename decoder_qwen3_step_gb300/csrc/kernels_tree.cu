// kernels_tree.cu - draft trees over the paged KV cache: rotary tables, the
// rotated append, the commit of an accepted path, and the merge of split
// attention.  (Attention itself: kernels_tree_f32.cu, kernels_tree_f16.cu,
// kernels_tree_tc.cu.)
#include <limits.h>

#include "tree_common.cuh"

namespace dec {

namespace {

// ---- rotary table ---------------------------------------------------------------
// (cos, sin)(p * freq_j) * mult.  The angle and its functions are formed in
// 64 bits and rounded once: at position 40,959 a 32-bit angle would be off by
// up to 2e-3.  Runs once per table.
__global__ void k_rope_table(const __grid_constant__ RopeTableArgs a) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.positions * a.pairs) return;
  double sn, cs;
  sincos((double)(i / a.pairs) * a.freq[i % a.pairs], &sn, &cs);
  reinterpret_cast<float2*>(a.table)[i] = make_float2((float)(cs * a.mult), (float)(sn * a.mult));
}

// ---- append ----------------------------------------------------------------------
// y = x / sqrt(mean x^2 + eps) * gain (queries and keys, when a gain is given);
// then for each pair (a, b) of the first rot channels
//   a' = a cos - b sin,  b' = b cos + a sin;
// queries go to q_out, keys and values to slot ctx + i of node i's sequence.
// One pass over the data, so HBM bounds it: D/4 lanes share a head row with four
// consecutive channels each (16-byte loads of fp32, 8 of 16-bit types) and take U
// heads of one node, all queries, all keys or all values, so that the node's
// angles and the gain are read once for them.  The pair's other channel is in the
// same lane (interleaved) or rot/8 lanes away (halves), one shuffle.
template <int D, int U, typename T>
__global__ void __launch_bounds__(256, U == 4 && sizeof(T) == 4 ? 5 : 4) k_tree_append(const __grid_constant__ TreeAppendArgs a) {
  constexpr int kLanes = D / 4, kSlots = 256 / kLanes;
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return;
  const int H = a.q ? a.d.H : 0, Hkv = a.k ? a.d.Hkv : 0, cq = (H + U - 1) / U, ck = (Hkv + U - 1) / U;
  const int lane = threadIdx.x % kLanes, el = lane * 4, half = a.rot >> 1;
  const uint32_t id = blockIdx.x * kSlots + threadIdx.x / kLanes, per = cq + 2 * ck;
  const int node = min((int)(id / per), a.m.N - 1), c = id % per;
  const bool live = id / per < (uint32_t)a.m.N;  // lanes behind the last node stay for the shuffles
  const bool is_q = c < cq, is_v = c >= cq + ck;
  const int h0 = (is_q ? c : is_v ? c - cq - ck : c - cq) * U, heads = is_q ? H : Hkv;
  const T* src = reinterpret_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) +
                  node * (is_q ? a.ldq : is_v ? a.ldv : a.ldk) + h0 * D + el;
  int pos = __ldg(a.m.pos + node);
  const int dst = __ldg(a.m.dst + node);
  float4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) x[u] = tree_load4(src + min(u, heads - 1 - h0) * D);
  const float* gain = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
  const float4 g = gain ? *reinterpret_cast<const float4*>(gain + el) : make_float4(1.f, 1.f, 1.f, 1.f);
  const bool pad = pos < 0;
  if (a.rope && pos >= a.rope_positions) {  // a replay whose plan outgrew the table of its capture
    if (lane == 0) atomicOr(a.m.err, kErrBounds);
    pos = a.rope_positions - 1;
  }
  const bool turn = a.rope && el < a.rot && !is_v && !pad;
  const bool first = el < half;  // halves: this lane's channels are the pairs' first
  float4 c0 = make_float4(1.f, 0.f, 1.f, 0.f), c1 = c0;  // (cos, sin) of the lane's pairs: four, or two when interleaved
  if (turn) {
    const float4* t = reinterpret_cast<const float4*>(a.rope + (size_t)pos * a.rot + (a.interleaved ? el : (first ? el : el - half) * 2));
    c0 = t[0];
    if (!a.interleaved) c1 = t[1];
  }
  const int other = turn ? (first ? lane + (half >> 2) : lane - (half >> 2)) : lane;
  const float sg = first ? -1.f : 1.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float4 y = x[u];
    if (a.q_norm || a.k_norm) {
      float ss = y.x * y.x + y.y * y.y + y.z * y.z + y.w * y.w;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rn = gain ? 1.0f / sqrtf(ss / (float)D + a.d.eps) : 1.f;
      y = make_float4(y.x * (rn * g.x), y.y * (rn * g.y), y.z * (rn * g.z), y.w * (rn * g.w));
    }
    if (a.rope) {
      if (a.interleaved) {
        if (turn)  // a product with sin = 0 would carry a channel that is not finite into its neighbour
          y = make_float4(y.x * c0.x - y.y * c0.y, y.y * c0.x + y.x * c0.y, y.z * c0.z - y.w * c0.w, y.w * c0.z + y.z * c0.w);
      } else {
        float4 p;
        p.x = __shfl_sync(0xffffffffu, y.x, other, kLanes);
        p.y = __shfl_sync(0xffffffffu, y.y, other, kLanes);
        p.z = __shfl_sync(0xffffffffu, y.z, other, kLanes);
        p.w = __shfl_sync(0xffffffffu, y.w, other, kLanes);
        if (turn)
          y = make_float4(y.x * c0.x + sg * p.x * c0.y, y.y * c0.z + sg * p.y * c0.w, y.z * c1.x + sg * p.z * c1.y,
                          y.w * c1.z + sg * p.w * c1.w);
      }
    }
    if (!live || h0 + u >= heads) continue;
    if (is_q) {
      // a padding node's query is zero: attention on it reads defined numbers
      tree_store4(a.q_out, a.q_type, node * a.ldo + (h0 + u) * D + el, pad ? make_float4(0.f, 0.f, 0.f, 0.f) : y);
    } else if (!pad) {
      const int64_t off = kv_offset(a.layer, dst >> 4, is_v, h0 + u, dst & 15, a.d.n_blocks, a.d.Hkv, 16, D);
      tree_store4(a.kv, a.kv_f16 ? kTreeF16 : kTreeF32, off + el, y);
    }
  }
}

template <int D, int U>
cudaError_t append_u(const TreeAppendArgs& a, cudaStream_t s) {
  constexpr int kSlots = 256 / (D / 4);
  const int64_t units = (int64_t)a.m.N * ((a.q ? (a.d.H + U - 1) / U : 0) + (a.k ? 2 * ((a.d.Hkv + U - 1) / U) : 0));
  const int grid = (int)((units + kSlots - 1) / kSlots);
  return a.in_type == kTreeF32   ? launch_pdl(k_tree_append<D, U, float>, grid, 256, 0, s, a)
         : a.in_type == kTreeF16 ? launch_pdl(k_tree_append<D, U, __half>, grid, 256, 0, s, a)
                                 : launch_pdl(k_tree_append<D, U, bf16>, grid, 256, 0, s, a);
}
template <int D>
cudaError_t append_d(const TreeAppendArgs& a, cudaStream_t s) {
  // a head per lane group while that leaves SMs idle: at 16:8 heads x 128, 16 nodes 1.8 us against 3.0 with four, 200 nodes
  // 3.4 with either, 1000 nodes 9.7 against 7.0
  const int64_t rows = (int64_t)a.m.N * ((a.q ? a.d.H : 0) + (a.k ? 2 * a.d.Hkv : 0));
  return rows <= 4ll * a.sms * (256 / (D / 4)) ? append_u<D, 1>(a, s) : append_u<D, 4>(a, s);
}

// ---- commit ----------------------------------------------------------------------
// The walk: from the root (taken as certain, or as prior chose) down to the
// child whose token is the one the model chose at its parent, the lowest such
// node, until there is none.  Then the K/V rows of the i-th node of the path
// move from slot ctx + path[i] to ctx + i in every layer.  path[i] >= i and
// path increases, so a row is never written before it has been read when the
// rows move in order; each thread owns 16 bytes of the row of one (layer,
// K or V, head) and moves them for the whole path, eight loads in flight, so
// no two threads ever touch the same bytes.  Every block repeats the walk (a
// few hundred loads) instead of waiting for another.
constexpr int kCommitThreads = 256;

__global__ void __launch_bounds__(kCommitThreads) k_tree_commit(const __grid_constant__ TreeCommitArgs a, int cols,
                                                                int blocks_per_seq) {
  __shared__ int child[kTreeMaxNodes + 1], path[kTreeMaxNodes], n_path;
  const int s = blockIdx.x / blocks_per_seq, part = blockIdx.x % blocks_per_seq;
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  const int b = __ldg(a.m.seq_start + s), T = min(__ldg(a.m.seq_start + s + 1) - b, kTreeMaxNodes);
  for (int i = threadIdx.x; i <= T; i += kCommitThreads) child[i] = INT_MAX;
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return;
  __syncthreads();
  for (int i = threadIdx.x; i < T; i += kCommitThreads) {
    const int p = __ldg(a.m.parents + b + i);
    if (p < -1) continue;  // padding
    const bool ok = p >= 0 ? a.draft[b + i] == a.target[b + p] : !a.prior || a.draft[b + i] == a.prior[s];
    if (ok) atomicMin(&child[p + 1], i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    for (int at = child[0]; at != INT_MAX; at = child[at + 1]) path[n++] = at;
    n_path = n;
  }
  __syncthreads();
  const int n = n_path;
  if (part == 0) {
    for (int i = threadIdx.x; i < T; i += kCommitThreads) a.path[b + i] = i < n ? path[i] : -1;
    if (threadIdx.x == 0) {
      a.accepted[s] = n;
      a.next[s] = n ? a.target[b + path[n - 1]] : a.prior ? a.prior[s] : -1;
    }
  }
  const int row_chunks = a.d.D * a.kv_bytes / 16;  // 16-byte pieces of a head row
  const int col = part * kCommitThreads + threadIdx.x;
  if (col >= cols) return;
  const int c = col % row_chunks, h = col / row_chunks % a.d.Hkv, lv = col / row_chunks / a.d.Hkv;
  const int64_t slab = (int64_t)a.d.Hkv * 16 * row_chunks;  // pieces of one (layer, block, K or V)
  int4* base = reinterpret_cast<int4*>(a.kv) + ((int64_t)(lv >> 1) * a.d.n_blocks * 2 + (lv & 1)) * slab +
               (int64_t)h * 16 * row_chunks + c;
  auto at = [&](int node) {
    const int d = __ldg(a.m.dst + b + node);
    return base + (int64_t)(d >> 4) * 2 * slab + (d & 15) * row_chunks;
  };
  int i0 = 0;
  while (i0 < n && path[i0] == i0) ++i0;  // already in place
  for (; i0 < n; i0 += 8) {
    int4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u < n) v[u] = *at(path[i0 + u]);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u < n) *at(i0 + u) = v[u];
  }
}

// ---- merge of split attention --------------------------------------------------------
// A unit whose keys several CTAs shared: with each CTA's running maximum m_c
// (base-2 logarithms), sum l_c and unnormalised output O_c,
//   out = sum_c O_c 2^(m_c - M) / sum_c l_c 2^(m_c - M),  M = max_c m_c.
// kWarps warps share a row, each adding every kWarps-th contribution in CTA
// order, then the warps' sums in warp order.  With four, the 38 records of a
// unit that 38 CTAs shared are two rounds of loads instead of ten.
template <int D, int kWarps>
__global__ void __launch_bounds__(128) k_tree_merge(const __grid_constant__ TreeAttendArgs a) {
  constexpr int kPer = D / 32, kRows = 4 / kWarps;
  __shared__ float part[kWarps == 1 ? 1 : 4][D + 1];
  const int R = a.m.row_tile, gs = a.d.gs, G = 1 << gs, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = R / kRows;
  TreeMerge e = a.m.merges[blockIdx.x / groups];  // the plan is older than the kernels before this one
  const int n = __ldg(a.m.hdr + kHdrMerges);
  const bool ok = tree_shape_ok(a.m, true);
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return;
  for (int w = blockIdx.x; w < n * groups; w += gridDim.x) {
    if (w != blockIdx.x) e = a.m.merges[w / groups];
    const int r = (w % groups) * kRows + warp / kWarps, c_first = warp % kWarps;
    const int row = e.row_tile * R + r, n_rec = (e.c1 - e.c0) / e.stride + 1;
    if (row >= e.nodes << gs) continue;  // with four warps a row, the whole block
    const int node = e.node0 + (row >> gs);
    auto rec = [&](int c) -> const float* { return tree_record(a, e.c0 + c * e.stride, c == 0); };
    const bool pad = __ldg(a.m.pos + node) < 0;
    float M = -INFINITY;
    for (int c = lane; c < n_rec; c += 32) M = fmaxf(M, __ldcg(rec(c) + R * D + r));
    M = warp_max(M);
    if (M == -INFINITY) M = 0.f;  // no contribution saw a finite score
    float L = 0.f, o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.f;
#pragma unroll 8
    for (int c = c_first; c < n_rec; c += kWarps) {
      const float* p = rec(c);
      const float f = ex2(__ldcg(p + R * D + r) - M);
      L = fmaf(__ldcg(p + R * D + R + r), f, L);
      if constexpr (kPer == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p + r * D + lane * 4));
        o[0] = fmaf(v.x, f, o[0]);
        o[1] = fmaf(v.y, f, o[1]);
        o[2] = fmaf(v.z, f, o[2]);
        o[3] = fmaf(v.w, f, o[3]);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[j] = fmaf(__ldcg(p + r * D + lane * kPer + j), f, o[j]);
      }
    }
    if constexpr (kWarps > 1) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) part[warp][lane * kPer + j] = o[j];
      if (lane == 0) part[warp][D] = L;
      __syncthreads();
      L = 0.f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        L += part[x][D];
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[j] += part[x][lane * kPer + j];
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const bool zero = pad || L == 0.f;
    const float inv = 1.0f / L;
    const int64_t off = node * a.ldo + (int64_t)(e.head * G + (row & (G - 1))) * D + lane * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = zero ? 0.f : o[j] * inv;
    if constexpr (kPer == 4) {
      tree_store4(a.out, a.out_type, off, make_float4(o[0], o[1], o[2], o[3]));
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) tree_store(a.out, a.out_type, off + j, o[j]);
    }
  }
}
template <int D>
cudaError_t merge_rows(const TreeAttendArgs& a, int n_merges, int parts, cudaStream_t s) {
  // four warps a row, or one: 1 sequence x 8 nodes over 4000 keys (38 parts a unit) 11.7 us, 18.0; 4 x 8 over 2000 (10 parts)
  // 12.4, 13.5; 16 x 8 over 1000 (3 parts) 19.1, 17.3; 32 x 8 over 1024-2048 (2 parts) 42.2, 38.1
  if (parts >= 8) return launch_pdl(k_tree_merge<D, 4>, n_merges * a.m.row_tile, 128, 0, s, a);
  return launch_pdl(k_tree_merge<D, 1>, n_merges * (a.m.row_tile / 4), 128, 0, s, a);
}

// The same for the row tiles of wide trees (128 or 256 rows), whose records
// are channel-major ([D/4][R] of four channels, then maxima and sums): thread =
// row, kC channels per block, so the reads are whole lines.  kG groups of 128
// threads share the records of a row.
template <int D, int kC, int kG>
__global__ void __launch_bounds__(128 * kG) k_tree_merge_wide(const __grid_constant__ TreeAttendArgs a) {
  constexpr int kSlabs = D / kC;
  __shared__ float top[kG][128], sum[kG][128];
  __shared__ float4 part[kG == 1 ? 1 : kG][kC / 4][128];
  const int gs = a.d.gs, R = a.m.row_tile, per = kSlabs * (R / 128), grp = threadIdx.x >> 7, t = threadIdx.x & 127;
  TreeMerge e = a.m.merges[blockIdx.x / per];  // the plan is older than the kernels before this one
  const int n = __ldg(a.m.hdr + kHdrMerges);
  const bool ok = tree_shape_ok(a.m, true);
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return;
  for (int w = blockIdx.x; w < n * per; w += gridDim.x) {
    if (w != blockIdx.x) e = a.m.merges[w / per];
    const int d0 = (w % kSlabs) * kC, r = (w % per) / kSlabs * 128 + t, row = e.row_tile * R + r;
    const int node = e.node0 + min(row >> gs, e.nodes - 1), n_rec = (e.c1 - e.c0) / e.stride + 1;
    auto rec = [&](int c) -> const float* { return tree_record(a, e.c0 + c * e.stride, c == 0); };
    const bool pad = __ldg(a.m.pos + node) < 0;
    float M = -INFINITY;
#pragma unroll 8
    for (int c = grp; c < n_rec; c += kG) M = fmaxf(M, __ldcg(rec(c) + R * D + r));
    if constexpr (kG > 1) {
      top[grp][t] = M;
      __syncthreads();
#pragma unroll
      for (int g = 0; g < kG; ++g) M = fmaxf(M, top[g][t]);
    }
    if (M == -INFINITY) M = 0.f;  // no contribution saw a finite score
    float L = 0.f;
    float4 o[kC / 4];
#pragma unroll
    for (int i = 0; i < kC / 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll kC == 4 ? 8 : 2
    for (int c = grp; c < n_rec; c += kG) {
      const float* p = rec(c);
      const float f = ex2(__ldcg(p + R * D + r) - M);
      L = fmaf(__ldcg(p + R * D + R + r), f, L);
#pragma unroll
      for (int i = 0; i < kC / 4; ++i) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p) + (d0 / 4 + i) * R + r);
        o[i].x = fmaf(v.x, f, o[i].x);
        o[i].y = fmaf(v.y, f, o[i].y);
        o[i].z = fmaf(v.z, f, o[i].z);
        o[i].w = fmaf(v.w, f, o[i].w);
      }
    }
    if constexpr (kG > 1) {
      sum[grp][t] = L;
#pragma unroll
      for (int i = 0; i < kC / 4; ++i) part[grp][i][t] = o[i];
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int g = 1; g < kG; ++g) {
          L += sum[g][t];
#pragma unroll
          for (int i = 0; i < kC / 4; ++i) {
            const float4 v = part[g][i][t];
            o[i] = make_float4(o[i].x + v.x, o[i].y + v.y, o[i].z + v.z, o[i].w + v.w);
          }
        }
      }
      __syncthreads();
    }
    if (grp > 0 || row >= e.nodes << gs) continue;
    const bool zero = pad || L == 0.f;
    const float inv = 1.0f / L;
    const int64_t off = node * a.ldo + (int64_t)((e.head << gs) + (row & ((1 << gs) - 1))) * D + d0;
#pragma unroll
    for (int i = 0; i < kC / 4; ++i)
      tree_store4(a.out, a.out_type, off + 4 * i,
                  zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv));
  }
}

template <int D>
cudaError_t merge_wide(const TreeAttendArgs& a, int n_merges, int parts, cudaStream_t s) {
  // many parts: four channels and four record groups per block, or too few loads are in flight for all those records
  // (1 sequence x 64 nodes over 8000 keys, 19 parts: 18.8 us against 30.9; 2 x 64 over 4000, 10 parts: 21.9 against 26.2; 4 x
  // 64 over 4000, 5 parts: 32.8 against 29.5)
  const int halves = a.m.row_tile / 128;
  if (parts >= 8) return launch_pdl(k_tree_merge_wide<D, 4, 4>, n_merges * halves * (D / 4), 512, 0, s, a);
  return launch_pdl(k_tree_merge_wide<D, 16, 1>, n_merges * halves * (D / 16), 128, 0, s, a);
}

// ---- test of the joins' flags --------------------------------------------------------
// Both sides of the flag of place 0 in one thread: the part first, or the wait until it runs out.
__global__ void k_tree_join_test(TreeMeta m, int late, uint64_t limit_ns) {
  if (!late) tree_publish(m, 0);
  tree_await(m, 0, limit_ns);
  tree_retire(m, 0);
  if (late) tree_publish(m, 0);
}

}  // namespace

cudaError_t launch_tree_join_test(const TreeMeta& m, int late, uint64_t limit_ns, cudaStream_t s) {
  k_tree_join_test<<<1, 1, 0, s>>>(m, late, limit_ns);
  return cudaGetLastError();
}

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t s) {
  k_rope_table<<<(a.positions * a.pairs + 255) / 256, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_append(const TreeAppendArgs& a, cudaStream_t s) {
  switch (a.d.D) {
    case 32: return append_d<32>(a, s);
    case 64: return append_d<64>(a, s);
    case 128: return append_d<128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t s) {
  const int cols = a.d.n_layers * 2 * a.d.Hkv * (a.d.D * a.kv_bytes / 16);
  const int per = (cols + kCommitThreads - 1) / kCommitThreads;
  return launch_pdl(k_tree_commit, a.m.S * per, kCommitThreads, 0, s, a, cols, per);
}

cudaError_t launch_tree_merge(const TreeAttendArgs& a, int n_merges, int parts, cudaStream_t s) {
  // a replayed call may meet a plan with more merges than at its capture: the blocks loop
  if (a.m.row_tile >= 128) {
    return a.d.D == 128 ? merge_wide<128>(a, max(n_merges, 1), parts, s) : merge_wide<64>(a, max(n_merges, 1), parts, s);
  }
  switch (a.d.D) {
    case 32: return merge_rows<32>(a, max(n_merges, 1), parts, s);
    case 64: return merge_rows<64>(a, max(n_merges, 1), parts, s);
    case 128: return merge_rows<128>(a, max(n_merges, 1), parts, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dec
