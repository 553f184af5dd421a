// kernels_q8.cu - a KV cache held in 8 bits: the append that quantises, the
// commit of an accepted path over pages with scales, and the reading back of
// keys and values (which serves every kind of cache).  The codes: q8.cuh; the
// attention: kernels_tree_q8.cu.
#include <algorithm>
#include <cfloat>

#include "q8.cuh"

namespace dec {

namespace {

// ---- append ----------------------------------------------------------------------
// Rows are formed as in k_tree_append (RMSNorm, rotation, fp32).  A page's scale
// needs the largest magnitude of all its rows first, so a warp takes the whole
// page: D/4 lanes share a row with four channels each, and up to 16 rows stay in
// registers (64 fp32 a lane at D = 128) between the maximum and the codes, one
// pass over the data.  Query rows go through the same code, `per` heads of a node
// a warp.  HBM bounds it: 8 KB of a warp's loads are in flight at once.
// Cached tokens of a page are read and written only where its e rises.
template <int D, int kKind, typename T>
__global__ void __launch_bounds__(256, 2) k_append_q8(const __grid_constant__ TreeAppendArgs a, int q_tasks, int per, int kv_warps) {
  constexpr int kLanes = D / 4, kRows = 32 / kLanes, kSteps = 16 / kRows;
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  const int n_pages = __ldg(a.m.hdr + kHdrPages);
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, el = (lane % kLanes) * 4, half = a.rot >> 1;
  const int warp = blockIdx.x * 8 + (threadIdx.x >> 5);
  const bool is_q = warp < q_tasks;
  const int kv_tasks = a.k ? n_pages * a.d.Hkv * 2 : 0, per_node = (a.d.H + per - 1) / per;
  // queries: one task; keys and values: every kv_warps-th, a replay may meet more pages than its capture
  for (int t = is_q ? 0 : warp - q_tasks; t < (is_q ? 1 : kv_tasks); t += is_q ? 1 : kv_warps) {
    const int h = is_q ? (warp % per_node) * per : t % a.d.Hkv;
    const bool is_v = !is_q && (t / a.d.Hkv & 1);
    int block = 0, node = warp / per_node, slot0 = 0, n = min(per, a.d.H - h);
    if (!is_q) {
      const int4 p = __ldg(reinterpret_cast<const int4*>(a.m.pages) + t / (2 * a.d.Hkv));
      block = p.x;
      node = p.y;
      slot0 = p.z;
      n = p.w;
    }
    const int64_t stride = is_q ? D : is_v ? a.ldv : a.ldk;  // between the task's rows
    const T* src = reinterpret_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) + node * (is_q ? a.ldq : stride) + h * D + el;
    float4 x[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (s * kRows < n) x[s] = tree_load4(src + min(s * kRows + sub, n - 1) * stride);
    int pos_of = __ldg(a.m.pos + node + (is_q ? 0 : min(lane & 15, n - 1)));  // row lane & 15's position
    if (a.rope && pos_of >= a.rope_positions) {  // a replay whose plan outgrew the table of its capture
      atomicOr(a.m.err, kErrBounds);
      pos_of = a.rope_positions - 1;
    }
    const float* gain = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
    const float4 g = gain ? *reinterpret_cast<const float4*>(gain + el) : make_float4(1.f, 1.f, 1.f, 1.f);
    const bool turns = a.rope && el < a.rot && !is_v, first = el < half;
    const int other = turns ? (first ? lane + (half >> 2) : lane - (half >> 2)) : lane;
    const float sg = first ? -1.f : 1.f;
    // (cos, sin) of the lane's pairs for row r: four, or two when interleaved
    auto angles = [&](int s, float4& c0, float4& c1) {
      const int pos = __shfl_sync(0xffffffffu, pos_of, min(s * kRows + sub, n - 1));
      c0 = c1 = make_float4(1.f, 0.f, 1.f, 0.f);
      if (turns && pos >= 0) {
        const float4* at = reinterpret_cast<const float4*>(a.rope + (size_t)pos * a.rot + (a.interleaved ? el : (first ? el : el - half) * 2));
        c0 = __ldg(at);
        if (!a.interleaved) c1 = __ldg(at + 1);
      }
    };
    float4 n0, n1;  // the next step's
    if (!is_v) angles(0, n0, n1);
    float amax = 0.f;
    bool odd = false;  // a value that is not finite
    uint32_t live = 0;  // bit s: the lane's row of step s is one and no padding
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s * kRows >= n) break;
      float4 y = x[s];
      const bool pad = __shfl_sync(0xffffffffu, pos_of, min(s * kRows + sub, n - 1)) < 0;
      if (!is_v) {
        const float4 c0 = n0, c1 = n1;
        if (!is_q && (s + 1) * kRows < n) angles(s + 1, n0, n1);
        if (gain) {
          float ss = y.x * y.x + y.y * y.y + y.z * y.z + y.w * y.w;
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float rn = 1.0f / sqrtf(ss / (float)D + a.d.eps);
          y = make_float4(y.x * (rn * g.x), y.y * (rn * g.y), y.z * (rn * g.z), y.w * (rn * g.w));
        }
        if (a.rope) {
          if (a.interleaved) {
            if (turns && !pad)  // a product with sin = 0 would carry a channel that is not finite into its neighbour
              y = make_float4(y.x * c0.x - y.y * c0.y, y.y * c0.x + y.x * c0.y, y.z * c0.z - y.w * c0.w, y.w * c0.z + y.z * c0.w);
          } else {
            float4 p;
            p.x = __shfl_sync(0xffffffffu, y.x, other, kLanes);
            p.y = __shfl_sync(0xffffffffu, y.y, other, kLanes);
            p.z = __shfl_sync(0xffffffffu, y.z, other, kLanes);
            p.w = __shfl_sync(0xffffffffu, y.w, other, kLanes);
            if (turns && !pad)
              y = make_float4(y.x * c0.x + sg * p.x * c0.y, y.y * c0.z + sg * p.y * c0.w, y.z * c1.x + sg * p.z * c1.y,
                              y.w * c1.z + sg * p.w * c1.w);
          }
        }
      }
      const int r = s * kRows + sub;
      if (is_q) {
        // a padding node's query is zero: attention on it reads defined numbers
        if (r < n) tree_store4(a.q_out, a.q_type, node * a.ldo + (h + r) * D + el, pad ? make_float4(0.f, 0.f, 0.f, 0.f) : y);
        continue;
      }
      if (r < n && !pad) {
        live |= 1u << s;
        const float m = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
        if (!(fabsf(y.x) <= FLT_MAX && fabsf(y.y) <= FLT_MAX && fabsf(y.z) <= FLT_MAX && fabsf(y.w) <= FLT_MAX)) {  // rare
          odd = true;
          for (float* v : {&y.x, &y.y, &y.z, &y.w}) {
            if (*v != *v) *v = 0.f;
            if (fabsf(*v) <= FLT_MAX) amax = fmaxf(amax, fabsf(*v));
          }
        } else {
          amax = fmaxf(amax, m);
        }
      }
      x[s] = y;
    }
    if (is_q) continue;
    amax = warp_max(amax);
    float* scale = a.scales + q8_scale_at(a.d, a.layer, block, h, is_v);
    uint8_t* page = reinterpret_cast<uint8_t*>(a.kv) + kv_offset(a.layer, block, is_v, h, 0, a.d.n_blocks, a.d.Hkv, 16, D) + el;
    int e = q8_need<kKind>(amax);
    if (slot0 > 0) {  // the page holds cached tokens
      const int was = q8_exp(*scale);
      if (e > was) {
        const float f = q8_two(was - e);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int r = s * kRows + sub;
          if (r >= slot0) break;
          uint32_t* w = reinterpret_cast<uint32_t*>(page + r * D);
          const float4 v = q8_unpack<kKind>(*w);
          *w = q8_pack<kKind>(make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        }
      }
      e = max(e, was);
      __syncwarp();  // every lane has the scale that was
    }
    const float inv = q8_two(-e);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (live >> s & 1u)
        *reinterpret_cast<uint32_t*>(page + (slot0 + s * kRows + sub) * D) =
            q8_pack<kKind>(make_float4(x[s].x * inv, x[s].y * inv, x[s].z * inv, x[s].w * inv));
    if (lane == 0) *scale = q8_two(e);
    if (odd) atomicOr(a.m.err, kErrNonFinite);
  }
}

template <int D, int kKind, typename T>
cudaError_t append_t(const TreeAppendArgs& a, cudaStream_t s) {
  // query rows a warp: one while that leaves SMs idle, 16 after
  const int per = (int64_t)a.m.N * a.d.H <= 32ll * a.sms ? 1 : 16;
  const int q_tasks = a.q ? a.m.N * ((a.d.H + per - 1) / per) : 0;
  const int kv_warps = a.k ? a.n_pages * a.d.Hkv * 2 : 0;
  return launch_pdl(k_append_q8<D, kKind, T>, (q_tasks + kv_warps + 7) / 8, 256, 0, s, a, q_tasks, per, (q_tasks + kv_warps + 7) / 8 * 8 - q_tasks);
}
template <int D, int kKind>
cudaError_t append_k(const TreeAppendArgs& a, cudaStream_t s) {
  return a.in_type == kTreeF32   ? append_t<D, kKind, float>(a, s)
         : a.in_type == kTreeF16 ? append_t<D, kKind, __half>(a, s)
                                 : append_t<D, kKind, bf16>(a, s);
}
template <int D>
cudaError_t append_d(const TreeAppendArgs& a, cudaStream_t s) {
  return a.kv_type == kTreeI8 ? append_k<D, kTreeI8>(a, s) : append_k<D, kTreeE4m3>(a, s);
}

// ---- commit ----------------------------------------------------------------------
// The walk is k_tree_commit's.  A warp takes one (layer, K or V, KV head) of a
// sequence and its pages from the first node's on: the rows that move to a page
// are loaded into registers (they come from this page or from later ones, whose
// rows are as they were: path[i] >= i), then e becomes what they need, at least
// what it was; if it rises the page's other rows are rounded again; then the rows
// are written.  A row that moves between pages of one scale keeps its codes.
constexpr int kCommitThreads = 256;

template <int D, int kKind>
__global__ void __launch_bounds__(kCommitThreads) k_commit_q8(const __grid_constant__ TreeCommitArgs a, int blocks_per_seq) {
  constexpr int kLanes = D / 4, kRows = 32 / kLanes, kSteps = 16 / kRows;
  __shared__ int child[kTreeMaxNodes + 1], path[kTreeMaxNodes], n_path;
  const int s = blockIdx.x / blocks_per_seq, part = blockIdx.x % blocks_per_seq;
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  const int b = __ldg(a.m.seq_start + s), T = min(__ldg(a.m.seq_start + s + 1) - b, kTreeMaxNodes);
  const int ctx = __ldg(&a.m.reads[s].ctx), tab = __ldg(&a.m.reads[s].tab);
  const int n = tree_walk<kCommitThreads>(a, s, b, T, ok, part == 0, child, path, &n_path);
  const int col = part * (kCommitThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31, sub = lane / kLanes, el = (lane % kLanes) * 4;
  if (col >= a.d.n_layers * 2 * a.d.Hkv) return;
  const int h = col % a.d.Hkv, is_v = col / a.d.Hkv & 1, layer = col / a.d.Hkv / 2;
  auto page_of = [&](int block) {
    return reinterpret_cast<uint8_t*>(a.kv) + kv_offset(layer, block, is_v, h, 0, a.d.n_blocks, a.d.Hkv, 16, D) + el;
  };
  auto scale_of = [&](int block) { return a.scales + q8_scale_at(a.d, layer, block, h, is_v); };
  int i0 = 0;
  while (i0 < n && path[i0] == i0) ++i0;  // already in place
  for (int p = (ctx + i0) >> 4; i0 < n && p <= (ctx + n - 1) >> 4; ++p) {
    const int block = __ldg(a.m.tables + tab + p);
    uint32_t w[kSteps], move = 0;
    float f[kSteps], amax = 0.f;  // the sources' scales
    const int was = q8_exp(*scale_of(block));
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int i = p * 16 + t * kRows + sub - ctx;  // the slot's node
      w[t] = 0;
      f[t] = 1.f;
      if (i < 0 || i >= n || path[i] == i) continue;
      const int d = __ldg(a.m.dst + b + path[i]);
      w[t] = *reinterpret_cast<const uint32_t*>(page_of(d >> 4) + (d & 15) * D);
      f[t] = q8_two(q8_exp(*scale_of(d >> 4)));
      move |= 1u << t;
    }
    if (!__any_sync(0xffffffffu, move != 0)) continue;
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      if (!(move >> t & 1u)) continue;
      const float4 v = q8_unpack<kKind>(w[t]);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))) * f[t]);
    }
    amax = warp_max(amax);  // every lane's loads are behind it
    const int e = max(q8_need<kKind>(amax), was);
    const float inv = q8_two(-e);
    uint8_t* page = page_of(block);
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int r = t * kRows + sub;
      uint32_t* at = reinterpret_cast<uint32_t*>(page + r * D);
      const bool stays = p * 16 + r - ctx < n && !(move >> t & 1u);
      if (stays && e > was) {
        w[t] = *at;
        f[t] = q8_two(was);
      }
      if ((move >> t & 1u) || (stays && e > was)) {
        const float4 v = q8_unpack<kKind>(w[t]);
        const float g = f[t] * inv;
        *at = q8_pack<kKind>(make_float4(v.x * g, v.y * g, v.z * g, v.w * g));
      }
    }
    __syncwarp();
    if (lane == 0) *scale_of(block) = q8_two(e);
    __syncwarp();  // the next page's rows may come from where other lanes look the scale up
  }
}

template <int D>
cudaError_t commit_d(const TreeCommitArgs& a, cudaStream_t s) {
  const int per = (a.d.n_layers * 2 * a.d.Hkv * 32 + kCommitThreads - 1) / kCommitThreads;
  return a.kv_type == kTreeI8 ? launch_pdl(k_commit_q8<D, kTreeI8>, a.m.S * per, kCommitThreads, 0, s, a, per)
                              : launch_pdl(k_commit_q8<D, kTreeE4m3>, a.m.S * per, kCommitThreads, 0, s, a, per);
}

// ---- reading back ------------------------------------------------------------------
// A warp per page: its 16 rows in 16-byte loads, all in flight, then the values in
// the output's type.  Neighbouring warps take neighbouring heads, whose rows lie
// side by side in the output.  HBM bounds it, the output's bytes most of all.
template <int D, int kType>
__global__ void __launch_bounds__(256) k_tree_read(const __grid_constant__ TreeReadArgs a, int64_t warps, bool wide) {
  constexpr int kSize = kType == kTreeF32 ? 4 : kType == kTreeF16 ? 2 : 1, kE = 16 / kSize, kLoads = 16 * D / (32 * kE) > 0 ? 16 * D / (32 * kE) : 1;
  static_assert(16 * D >= 32 * kE, "a page is a load of every lane at least");
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  const int S = a.m.S, nb = __ldg(&a.m.reads[S].blocks[a.part]);
  const bool fits = __ldg(a.m.hdr + kHdrRows + a.part) == a.rows;
  if (ok && !fits && threadIdx.x == 0) atomicOr(a.m.err, kErrShape);
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok || !fits) return;
  const int lane = threadIdx.x & 31, sides = (a.k ? 1 : 0) + (a.v ? 1 : 0);
  const int64_t tasks = (int64_t)a.n_layers * nb * sides * a.d.Hkv;
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < tasks; t += warps) {
    const int h = t % a.d.Hkv, side = t / a.d.Hkv % sides, is_v = a.k ? side : 1;
    const int64_t lb = t / a.d.Hkv / sides;
    const int b = lb % nb, layer = lb / nb;
    int s = 0;  // the last sequence with reads[s].blocks <= b has it (those without blocks are passed over)
    for (int hi = S; hi - s > 1;) {
      const int mid = (s + hi) >> 1;
      if (__ldg(&a.m.reads[mid].blocks[a.part]) <= b) s = mid;
      else hi = mid;
    }
    const TreeReadSeq& q = a.m.reads[s];
    const int ctx = __ldg(&q.ctx), from = a.part ? ctx >> 4 : 0, p = from + b - __ldg(&q.blocks[a.part]);
    const int rows = min(16, ctx + __ldg(&q.nodes) - p * 16), block = __ldg(a.m.tables + __ldg(&q.tab) + p);
    const int64_t row0 = __ldg(&q.rows[a.part]) + (p - from) * 16;
    const uint8_t* page = reinterpret_cast<const uint8_t*>(a.kv) + kv_offset(a.layer + layer, block, is_v, h, 0, a.d.n_blocks, a.d.Hkv, 16, D) * kSize;
    float f = 1.f;
    if constexpr (kSize == 1) f = a.scales[q8_scale_at(a.d, a.layer + layer, block, h, is_v)];
    uint4 raw[kLoads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l) raw[l] = *reinterpret_cast<const uint4*>(page + (l * 32 + lane) * 16);
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int i = (l * 32 + lane) * kE, r = i / D;
      if (r >= rows) continue;
      const uint32_t w[4] = {raw[l].x, raw[l].y, raw[l].z, raw[l].w};
      float4 v[kE / 4];
#pragma unroll
      for (int j = 0; j < kE / 4; ++j) {
        if constexpr (kType == kTreeF32) {
          v[j] = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
        } else if constexpr (kType == kTreeF16) {
          const float2 x = tree_pair<__half>(w[2 * j]), y = tree_pair<__half>(w[2 * j + 1]);
          v[j] = make_float4(x.x, x.y, y.x, y.y);
        } else {
          const float4 c = q8_unpack<kType>(w[j]);
          v[j] = make_float4(c.x * f, c.y * f, c.z * f, c.w * f);
        }
      }
      void* out = is_v ? a.v : a.k;
      const int64_t at = layer * a.layer_stride + (row0 + r) * a.ld + h * D + i % D;
      if (kE > 4 && wide && a.out_type != kTreeF32) {
#pragma unroll
        for (int j = 0; j + 1 < kE / 4; j += 2) {
          const float z[8] = {v[j].x, v[j].y, v[j].z, v[j].w, v[j + 1].x, v[j + 1].y, v[j + 1].z, v[j + 1].w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (a.out_type == kTreeF16) {
              const __half2 y = __floats2half2_rn(z[2 * k], z[2 * k + 1]);
              o[k] = *reinterpret_cast<const uint32_t*>(&y);
            } else {
              const __nv_bfloat162 y = __floats2bfloat162_rn(z[2 * k], z[2 * k + 1]);
              o[k] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + at + j * 4) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kE / 4; ++j) tree_store4(out, a.out_type, at + j * 4, v[j]);
      }
    }
  }
}

template <int D>
cudaError_t read_d(const TreeReadArgs& a, cudaStream_t s) {
  const int64_t tasks = (int64_t)a.n_layers * a.n_blocks * ((a.k ? 1 : 0) + (a.v ? 1 : 0)) * a.d.Hkv;
  const int grid = (int)std::min<int64_t>((tasks + 7) / 8, 1 << 20);
  const bool wide = (((uintptr_t)a.k | (uintptr_t)a.v) & 15) == 0 && a.ld % 8 == 0 && a.layer_stride % 8 == 0;  // 16-byte pieces
  switch (a.kv_type) {
    case kTreeF32: return launch_pdl(k_tree_read<D, kTreeF32>, grid, 256, 0, s, a, (int64_t)grid * 8, wide);
    case kTreeF16: return launch_pdl(k_tree_read<D, kTreeF16>, grid, 256, 0, s, a, (int64_t)grid * 8, wide);
    case kTreeE4m3: return launch_pdl(k_tree_read<D, kTreeE4m3>, grid, 256, 0, s, a, (int64_t)grid * 8, wide);
    default: return launch_pdl(k_tree_read<D, kTreeI8>, grid, 256, 0, s, a, (int64_t)grid * 8, wide);
  }
}

}  // namespace

cudaError_t launch_tree_append_q8(const TreeAppendArgs& a, cudaStream_t s) {
  return a.d.D == 32 ? append_d<32>(a, s) : a.d.D == 64 ? append_d<64>(a, s) : append_d<128>(a, s);
}
cudaError_t launch_tree_commit_q8(const TreeCommitArgs& a, cudaStream_t s) {
  return a.d.D == 32 ? commit_d<32>(a, s) : a.d.D == 64 ? commit_d<64>(a, s) : commit_d<128>(a, s);
}
cudaError_t launch_tree_read(const TreeReadArgs& a, cudaStream_t s) {
  return a.d.D == 32 ? read_d<32>(a, s) : a.d.D == 64 ? read_d<64>(a, s) : read_d<128>(a, s);
}

}  // namespace dec
