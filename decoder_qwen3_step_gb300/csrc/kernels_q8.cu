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
// page: D/4 lanes share a row with four channels each, and the formed rows wait in
// shared memory (8 KB a warp at D = 128) between the maximum and the codes, one
// pass over the data.  Query rows go through the same code, `per` heads of a node
// a warp.
// Large calls are bound by latency: 20 warps an SM, one task each, copy, wait for
// all of it and work (32 x 256 nodes: 195 MB in 50 us, 3.9 TB/s, 44% of the issue
// slots, 26% of the warps).  A task's rows are copied to shared memory all at once
// (with four steps of them in flight 56 us; with the rows in registers, every loop
// unrolled to 16 rows and 147 instructions a row, 82), and the loops go four steps at a time: their
// sums of squares are reduced together (6 shuffles for 4 rows of 128 channels; the
// lanes end up with one row's each, so one root and quotient serve four rows), and
// what is rare is looked for once a page (padding, values that are not finite, e
// at its end).
// Cached tokens of a page are read and written only where its e rises.
constexpr int kAppendSide = 4;  // steps of rows at a time

// 8 or 16 bytes global -> shared, waited for by the thread that asked.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(kBytes) : "memory");
}

// Codes of four values times inv = 2^-e where the largest magnitude is known to fit.
template <int kKind>
__device__ __forceinline__ uint32_t q8_pack_fit(float4 y, float inv) {
  if constexpr (Q8<kKind>::kInt) {  // 1.5 2^23 + code: rounded to a whole number, its last byte is the code
    constexpr float k = 12582912.f;
    const uint32_t a = __byte_perm(__float_as_uint(fmaf(y.x, inv, k)), __float_as_uint(fmaf(y.y, inv, k)), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(fmaf(y.z, inv, k)), __float_as_uint(fmaf(y.w, inv, k)), 0x0040);
    return __byte_perm(a, b, 0x5410);
  } else {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(y.x * inv, y.y * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(y.z * inv, y.w * inv), __NV_SATFINITE, __NV_E4M3);
    return a | (b << 16);
  }
}

template <int D, int kKind, typename T>
__global__ void __launch_bounds__(128, 5) k_append_q8(const __grid_constant__ TreeAppendArgs a, int q_tasks, int per, int kv_warps) {
  constexpr int kLanes = D / 4, kRows = 32 / kLanes, kSide = kAppendSide;
  extern __shared__ __align__(16) float4 formed[];  // [4 warps][16 rows][kLanes]
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  const int n_pages = __ldg(a.m.hdr + kHdrPages);
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, li = lane % kLanes, el = li * 4, half = a.rot >> 1;
  const int warp = blockIdx.x * 4 + (threadIdx.x >> 5);
  float4* rows = formed + (threadIdx.x >> 5) * 16 * kLanes + li;
  const bool is_q = warp < q_tasks;
  const int kv_tasks = a.k ? n_pages * a.d.Hkv * 2 : 0, per_node = (a.d.H + per - 1) / per;
  // queries: one task; keys and values: every kv_warps-th, a replay may meet more pages than its capture
  for (int t = is_q ? 0 : warp - q_tasks; t < (is_q ? 1 : kv_tasks); t += is_q ? 1 : kv_warps) {
    const int h = is_q ? (warp % per_node) * per : t % a.d.Hkv;
    const bool is_v = !is_q && (t / a.d.Hkv & 1);
    int block = 0, node = warp / per_node, slot0 = 0, n = min(per, a.d.H - h);
    if (!is_q) {
      const int4 p = __ldg(reinterpret_cast<const int4*>(a.m.pages) + t / (2 * a.d.Hkv));
      block = tree_block(a.m, a.d.n_blocks, p.x);
      node = p.y;
      slot0 = p.z;
      n = p.w;
    }
    const int64_t stride = is_q ? D : is_v ? a.ldv : a.ldk;  // between the task's rows
    const T* src = reinterpret_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) + node * (is_q ? a.ldq : stride) + h * D + el;
    // every row of the task on its way to where its lane formed values go (four channels of a lane, no other lane's); rows
    // behind the last are the last again
#pragma unroll 4
    for (int s = 0; s * kRows < (n + kSide * kRows - 1) / (kSide * kRows) * (kSide * kRows); ++s)
      copy_async<4 * sizeof(T)>(rows + (s * kRows + sub) * kLanes, src + min(s * kRows + sub, n - 1) * stride);
    int pos_of = __ldg(a.m.pos + node + (is_q ? 0 : min(lane & 15, n - 1)));  // row lane & 15's position
    if (a.rope && pos_of >= a.rope_positions) {  // a replay whose plan outgrew the table of its capture
      atomicOr(a.m.err, kErrBounds);
      pos_of = a.rope_positions - 1;
    }
    const bool pads = __any_sync(0xffffffffu, pos_of < 0);
    auto pos_at = [&](int r) { return __shfl_sync(0xffffffffu, pos_of, min(r, n - 1)); };
    const float* gain = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
    const float4 g = gain ? *reinterpret_cast<const float4*>(gain + el) : make_float4(1.f, 1.f, 1.f, 1.f);
    const bool rope = a.rope && !is_v, turns = rope && el < a.rot, first = el < half;
    const int other = turns ? (first ? lane + (half >> 2) : lane - (half >> 2)) : lane;
    // (cos, sin) of the lane's pairs, four, or two when interleaved; halves: sin with the sign that the lane's channels take.
    // A query task has one position.
    float4 c0[kSide], c1[kSide];
    const float* at = a.rope + (a.interleaved ? el : (first ? el : el - half) * 2);
    auto angles = [&](int pos, float4& x, float4& y) {
      x = y = make_float4(1.f, 0.f, 1.f, 0.f);
      if (turns && pos >= 0) {
        const float4* p = reinterpret_cast<const float4*>(at + (size_t)pos * a.rot);
        x = __ldg(p);
        if (!a.interleaved) {
          y = __ldg(p + 1);
          if (first) x.y = -x.y, x.w = -x.w, y.y = -y.y, y.w = -y.w;
        }
      }
    };
    if (rope && is_q) {
      angles(pos_of, c0[0], c1[0]);
#pragma unroll
      for (int j = 1; j < kSide; ++j) c0[j] = c0[0], c1[j] = c1[0];
    }
    char* out = nullptr;  // queries: the lane's first row and the bytes between rows
    const int out_row = D * (a.q_type == kTreeF32 ? 4 : 2);
    if (is_q) out = reinterpret_cast<char*>(a.q_out) + (node * a.ldo + (h + sub) * D + el) * (a.q_type == kTreeF32 ? 4 : 2);
    float amax = 0.f, bad = 0.f;  // bad: NaN once a value is not finite
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
    for (int s0 = 0; s0 * kRows < n; s0 += kSide) {
      float4 x[kSide];
#pragma unroll
      for (int j = 0; j < kSide; ++j) x[j] = tree_load4(reinterpret_cast<const T*>(rows + ((s0 + j) * kRows + sub) * kLanes));
      if (rope && !is_q) {
#pragma unroll
        for (int j = 0; j < kSide; ++j) angles(pos_at((s0 + j) * kRows + sub), c0[j], c1[j]);
      }
      if (gain) {
        float ss[kSide];
#pragma unroll
        for (int j = 0; j < kSide; ++j) ss[j] = x[j].x * x[j].x + x[j].y * x[j].y + x[j].z * x[j].z + x[j].w * x[j].w;
        // lanes whose bit o is set go on with the upper half of the sums: after log2(kSide) exchanges a lane has one sum
        int o = kLanes / 2;
#pragma unroll
        for (int w = kSide / 2; w > 0; w /= 2, o /= 2) {
          const bool up = lane & o;
#pragma unroll
          for (int j = 0; j < w; ++j) {
            const float give = up ? ss[j] : ss[j + w], keep = up ? ss[j + w] : ss[j];
            ss[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
#pragma unroll
        for (; o > 0; o /= 2) ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], o);
        const float r = 1.0f / sqrtf(ss[0] / (float)D + a.d.eps);
#pragma unroll
        for (int j = 0; j < kSide; ++j) {
          const float rn = __shfl_sync(0xffffffffu, r, j * (kLanes / kSide), kLanes);
          x[j] = make_float4(x[j].x * (rn * g.x), x[j].y * (rn * g.y), x[j].z * (rn * g.z), x[j].w * (rn * g.w));
        }
      }
      if (rope) {
#pragma unroll
        for (int j = 0; j < kSide; ++j) {
          float4& y = x[j];
          // channels that are not turned stay as they are: a product with sin = 0 would carry one that is not finite into its pair
          if (a.interleaved) {
            if (turns)
              y = make_float4(y.x * c0[j].x - y.y * c0[j].y, y.y * c0[j].x + y.x * c0[j].y, y.z * c0[j].z - y.w * c0[j].w, y.w * c0[j].z + y.z * c0[j].w);
          } else {
            float4 p;
            p.x = __shfl_sync(0xffffffffu, y.x, other, kLanes);
            p.y = __shfl_sync(0xffffffffu, y.y, other, kLanes);
            p.z = __shfl_sync(0xffffffffu, y.z, other, kLanes);
            p.w = __shfl_sync(0xffffffffu, y.w, other, kLanes);
            if (turns)
              y = make_float4(y.x * c0[j].x + p.x * c0[j].y, y.y * c0[j].z + p.y * c0[j].w, y.z * c1[j].x + p.z * c1[j].y, y.w * c1[j].z + p.w * c1[j].w);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kSide; ++j) {
        const int r = (s0 + j) * kRows + sub;
        if (pads && pos_at(r) < 0) x[j] = make_float4(0.f, 0.f, 0.f, 0.f);  // a query of zeros: attention on it reads defined numbers
        if (is_q) {
          if (r < n) tree_store4(out + r / kRows * (kRows * out_row), a.q_type, 0, x[j]);
        } else {
          rows[r * kLanes] = x[j];
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[j].x), fabsf(x[j].y)), fmaxf(fabsf(x[j].z), fabsf(x[j].w))));
          bad = fmaf(x[j].x, 0.f, fmaf(x[j].y, 0.f, fmaf(x[j].z, 0.f, fmaf(x[j].w, 0.f, bad))));
        }
      }
    }
    if (is_q) continue;
    const bool odd = __any_sync(0xffffffffu, bad != 0.f);
    if (odd) {  // rare: the maximum of what is finite, NaN as 0
      amax = 0.f;
#pragma unroll 1
      for (int r = sub; r < n; r += kRows) {
        float4 y = rows[r * kLanes];
        for (float* v : {&y.x, &y.y, &y.z, &y.w}) {
          if (*v != *v) *v = 0.f;
          if (fabsf(*v) <= FLT_MAX) amax = fmaxf(amax, fabsf(*v));
        }
        rows[r * kLanes] = y;
      }
      if (lane == 0) atomicOr(a.m.err, kErrNonFinite);
    }
    amax = warp_max(amax);
    float* scale = a.scales + q8_scale_at(a.d, a.layer, block, h, is_v);
    uint8_t* page = reinterpret_cast<uint8_t*>(a.kv) + kv_offset(a.layer, block, is_v, h, 0, a.d.n_blocks, a.d.Hkv, 16, D) + el;
    int e = q8_need<kKind>(amax);
    if (slot0 > 0) {  // the page holds cached tokens
      const int was = q8_exp(*scale);
      if (e > was) {
        const float f = q8_two(was - e);
#pragma unroll 4
        for (int r = sub; r < slot0; r += kRows) {
          uint32_t* w = reinterpret_cast<uint32_t*>(page + r * D);
          const float4 v = q8_unpack<kKind>(*w);
          *w = q8_pack<kKind>(make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        }
      }
      e = max(e, was);
      __syncwarp();  // every lane has the scale that was
    }
    const float inv = q8_two(-e);
    page += slot0 * D;
    const bool fits = !odd && e < kExpMax;
#pragma unroll 4
    for (int s = 0; s * kRows < n; ++s) {  // each lane's own values
      const int r = s * kRows + sub;
      const bool pad = pads && pos_at(r) < 0;  // a shuffle: every lane, also those behind the last row
      if (r >= n || pad) continue;
      const float4 y = rows[r * kLanes];
      *reinterpret_cast<uint32_t*>(page + r * D) = fits ? q8_pack_fit<kKind>(y, inv) : q8_pack<kKind>(make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    }
    if (lane == 0) *scale = q8_two(e);
  }
}

template <int D, int kKind, typename T>
cudaError_t append_t(const TreeAppendArgs& a, cudaStream_t s) {
  static SmemOptIn opt;
  constexpr int smem = 4 * 16 * D * 4;
  cudaError_t e = opt.ensure(k_append_q8<D, kKind, T>, smem);
  if (e != cudaSuccess) return e;
  // query rows a warp: one while that leaves SMs idle, 16 after (32 x 17 nodes of 16 heads: 7.5 us, with four 11)
  const int per = (int64_t)a.m.N * a.d.H <= 20ll * a.sms ? 1 : 16;
  const int q_tasks = a.q ? a.m.N * ((a.d.H + per - 1) / per) : 0;
  const int kv_warps = a.k ? a.n_pages * a.d.Hkv * 2 : 0;
  const int grid = (q_tasks + kv_warps + 3) / 4;
  return launch_pdl(k_append_q8<D, kKind, T>, grid, 128, smem, s, a, q_tasks, per, grid * 4 - q_tasks);
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
// sequence and its pages from the first one on that a row moves to: the rows that
// move there are loaded into registers, 16 codes a lane (they come from this page
// or from later ones, whose rows are as they were: path[i] >= i), then e becomes
// what they need, at least what it was; if it rises the page's other rows are
// rounded again; then the rows are written.  Rows from pages of the same scale keep
// their codes (their values fit), a page that gets no others is a copy.
// Latency bounds it, not the few bytes; instructions come next (with four codes a
// lane, 16 steps a page, 32 sequences x 64 nodes over 28 layers took 24 us, so 12).
constexpr int kCommitThreads = 256;

template <int D, int kKind>
__global__ void __launch_bounds__(kCommitThreads, 4) k_commit_q8(const __grid_constant__ TreeCommitArgs a, int blocks_per_seq) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kSteps = 16 / kRows;
  __shared__ int child[kTreeMaxNodes + 1], path[kTreeMaxNodes], dst[kTreeMaxNodes], n_path;
  const int s = blockIdx.x / blocks_per_seq, part = blockIdx.x % blocks_per_seq;
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  const int b = __ldg(a.m.seq_start + s), T = min(__ldg(a.m.seq_start + s + 1) - b, kTreeMaxNodes);
  const int ctx = __ldg(&a.m.reads[s].ctx), tab = __ldg(&a.m.reads[s].tab);
  for (int i = threadIdx.x; ok && i < T; i += kCommitThreads) {  // (of another plan b may be anything)
    const int d = __ldg(a.m.dst + b + i);
    dst[i] = tree_block(a.m, a.d.n_blocks, d >> 4) * 16 + (d & 15);
  }
  const int n = tree_walk<kCommitThreads>(a, s, b, T, ok, part == 0, child, path, &n_path);
  const int lane = threadIdx.x & 31, sub = lane / kLanes, el = (lane % kLanes) * 16;
  int i0 = 0;
  while (i0 < n && path[i0] == i0) ++i0;  // already in place
  if (i0 == n) return;
  const int col = part * (kCommitThreads / 32) + (threadIdx.x >> 5);
  if (col >= a.d.n_layers * 2 * a.d.Hkv) return;
  const int h = col % a.d.Hkv, is_v = col / a.d.Hkv & 1, layer = col / a.d.Hkv / 2;
  auto page_of = [&](int block) {
    return reinterpret_cast<uint8_t*>(a.kv) + kv_offset(layer, block, is_v, h, 0, a.d.n_blocks, a.d.Hkv, 16, D) + el;
  };
  auto scale_of = [&](int block) { return a.scales + q8_scale_at(a.d, layer, block, h, is_v); };
  for (int p = (ctx + i0) >> 4; p <= (ctx + n - 1) >> 4; ++p) {
    const int block = tree_block(a.m, a.d.n_blocks, __ldg(a.m.tables + tab + p));
    uint8_t* page = page_of(block);
    uint4 w[kSteps];
    float f[kSteps];  // the sources' scales
    uint32_t move = 0;
    const int was = q8_exp(*scale_of(block));
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int i = p * 16 + t * kRows + sub - ctx;  // the slot's node
      const int from = i >= 0 && i < n ? path[i] : i;
      if (from != i) {
        const int d = dst[from];
        w[t] = *reinterpret_cast<const uint4*>(page_of(d >> 4) + (d & 15) * D);
        f[t] = *scale_of(d >> 4);
        move |= 1u << t;
      }
    }
    bool other = false;  // a row of another scale
#pragma unroll
    for (int t = 0; t < kSteps; ++t)
      if (move >> t & 1u) {
        f[t] = q8_two(q8_exp(f[t]));
        other |= f[t] != q8_two(was);
      }
    __syncwarp();  // every lane's rows and scales are loaded before any of them is written over
    if (!__any_sync(0xffffffffu, other)) {
#pragma unroll
      for (int t = 0; t < kSteps; ++t)
        if (move >> t & 1u) *reinterpret_cast<uint4*>(page + (t * kRows + sub) * D) = w[t];
      __syncwarp();  // other lanes read these rows, or this page's neighbours, next
      continue;
    }
    float amax = 0.f;
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      if (!(move >> t & 1u)) continue;
      const uint32_t c[4] = {w[t].x, w[t].y, w[t].z, w[t].w};
      float m = 0.f;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const float4 v = q8_unpack<kKind>(c[z]);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
      }
      amax = fmaxf(amax, m * f[t]);
    }
    amax = warp_max(amax);
    const int e = max(q8_need<kKind>(amax), was);
    const float inv = q8_two(-e);
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int r = t * kRows + sub;
      uint4* at = reinterpret_cast<uint4*>(page + r * D);
      const bool moves = move >> t & 1u, again = !moves && e > was && p * 16 + r - ctx < n;
      if (!moves && !again) continue;
      const uint4 x = again ? *at : w[t];
      const float g = (again ? q8_two(was) : f[t]) * inv;
      uint32_t c[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const float4 v = q8_unpack<kKind>(c[z]);
        c[z] = q8_pack_fit<kKind>(v, g);
      }
      *at = make_uint4(c[0], c[1], c[2], c[3]);
    }
    __syncwarp();
    if (lane == 0) *scale_of(block) = q8_two(e);
    __syncwarp();  // the next page's rows may come from where other lanes look the scale up
  }
}

template <int D>
cudaError_t commit_d(const TreeCommitArgs& a, cudaStream_t s) {
  const int per = (a.d.n_layers * 2 * a.d.Hkv * 32 + kCommitThreads - 1) / kCommitThreads;  // a column for every warp
  return a.kv_type == kTreeI8 ? launch_pdl(k_commit_q8<D, kTreeI8>, a.m.S * per, kCommitThreads, 0, s, a, per)
                              : launch_pdl(k_commit_q8<D, kTreeE4m3>, a.m.S * per, kCommitThreads, 0, s, a, per);
}

// ---- reading back ------------------------------------------------------------------
// A block of threads per pool block and layer, a warp per page (KV head, K or V):
// its 16 rows in 16-byte loads, all in flight, then the values in the output's
// type.  A block's warps fill whole rows of the output between them.  HBM bounds
// it, the output's bytes most of all: 28 layers of 32 x 1024-2048 tokens from i8 to
// f16 1328 us, 8.5 GB at 6.4 TB/s (with two pages a warp at a time 1728).
template <int D, int kType>
__global__ void __launch_bounds__(256) k_tree_read(const __grid_constant__ TreeReadArgs a, bool wide) {
  constexpr int kSize = kType == kTreeF32 ? 4 : kType == kTreeF16 ? 2 : 1, kE = 16 / kSize, kLoads = 16 * D / (32 * kE);
  static_assert(kLoads >= 1, "a page is a load of every lane at least");
  const bool ok = tree_shape_ok(a.m);  // the plan is older than the kernels before this one
  const int S = a.m.S, nb = __ldg(&a.m.reads[S].blocks[a.part]);
  const bool fits = __ldg(a.m.hdr + kHdrRows + a.part) == a.rows;
  if (ok && !fits && threadIdx.x == 0) atomicOr(a.m.err, kErrShape);
  // a block's sequence, entry and rows
  int s = 0, from = 0, p = 0, rows = 0, block = 0;
  int64_t row0 = 0;
  auto place = [&](int b) {
    s = 0;  // the last sequence with reads[s].blocks <= b has it (those without blocks are passed over)
    for (int hi = S; hi - s > 1;) {
      const int mid = (s + hi) >> 1;
      if (__ldg(&a.m.reads[mid].blocks[a.part]) <= b) s = mid;
      else hi = mid;
    }
    const TreeReadSeq& q = a.m.reads[s];
    const int ctx = __ldg(&q.ctx);
    from = a.part ? ctx >> 4 : 0;
    p = from + b - __ldg(&q.blocks[a.part]);
    rows = min(16, ctx + __ldg(&q.nodes) - p * 16);
    block = tree_block(a.m, a.d.n_blocks, __ldg(a.m.tables + __ldg(&q.tab) + p));
    row0 = __ldg(&q.rows[a.part]) + (p - from) * 16;
  };
  if (ok && fits && blockIdx.x < nb) place(blockIdx.x);
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok || !fits) return;
  const int lane = threadIdx.x & 31, pages = ((a.k ? 1 : 0) + (a.v ? 1 : 0)) * a.d.Hkv;
  for (int layer = blockIdx.y; layer < a.n_layers; layer += gridDim.y)
    for (int b = blockIdx.x; b < nb; b += gridDim.x) {
      if (gridDim.x < nb) place(b);
      for (int i = threadIdx.x >> 5; i < pages; i += 8) {
        const int h = i % a.d.Hkv, is_v = a.k ? i >= a.d.Hkv : 1;
        const uint8_t* page = reinterpret_cast<const uint8_t*>(a.kv) + kv_offset(a.layer + layer, block, is_v, h, 0, a.d.n_blocks, a.d.Hkv, 16, D) * kSize;
        const float f = kSize == 1 ? a.scales[q8_scale_at(a.d, a.layer + layer, block, h, is_v)] : 1.f;
        uint4 raw[kLoads];
#pragma unroll
        for (int l = 0; l < kLoads; ++l) raw[l] = *reinterpret_cast<const uint4*>(page + (l * 32 + lane) * 16);
        void* out = is_v ? a.v : a.k;
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          const int e = (l * 32 + lane) * kE, r = e / D;
          if (r >= rows) continue;
          const uint32_t w[4] = {raw[l].x, raw[l].y, raw[l].z, raw[l].w};
          float4 v[kE / 4];
#pragma unroll
          for (int j = 0; j < kE / 4; ++j) {
            if constexpr (kType == kTreeF32) {
              v[j] = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
            } else if constexpr (kType == kTreeF16) {
              const float2 g = tree_pair<__half>(w[2 * j]), z = tree_pair<__half>(w[2 * j + 1]);
              v[j] = make_float4(g.x, g.y, z.x, z.y);
            } else {
              const float4 c = q8_unpack<kType>(w[j]);
              v[j] = make_float4(c.x * f, c.y * f, c.z * f, c.w * f);
            }
          }
          const int64_t at = layer * a.layer_stride + (row0 + r) * a.ld + h * D + e % D;
          if (kE > 4 && wide && a.out_type != kTreeF32) {
#pragma unroll
            for (int j = 0; j + 1 < kE / 4; j += 2) {
              const float z[8] = {v[j].x, v[j].y, v[j].z, v[j].w, v[j + 1].x, v[j + 1].y, v[j + 1].z, v[j + 1].w};
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (a.out_type == kTreeF16) {
                  const __half2 x = __floats2half2_rn(z[2 * k], z[2 * k + 1]);
                  o[k] = *reinterpret_cast<const uint32_t*>(&x);
                } else {
                  const __nv_bfloat162 x = __floats2bfloat162_rn(z[2 * k], z[2 * k + 1]);
                  o[k] = *reinterpret_cast<const uint32_t*>(&x);
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
}

template <int D, int kType>
cudaError_t read_t(const TreeReadArgs& a, cudaStream_t s) {
  const bool wide = (((uintptr_t)a.k | (uintptr_t)a.v) & 15) == 0 && a.ld % 8 == 0 && a.layer_stride % 8 == 0;  // 16-byte pieces
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_blocks, std::min(a.n_layers, 65535));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_read<D, kType>, a, wide);
}
template <int D>
cudaError_t read_d(const TreeReadArgs& a, cudaStream_t s) {
  switch (a.kv_type) {
    case kTreeF32: return read_t<D, kTreeF32>(a, s);
    case kTreeF16: return read_t<D, kTreeF16>(a, s);
    case kTreeE4m3: return read_t<D, kTreeE4m3>(a, s);
    default: return read_t<D, kTreeI8>(a, s);
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
