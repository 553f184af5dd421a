// kernels_tree_f32.cu - tree attention over an fp32 cache (the parity mode):
// true fp32 products on the FFMA pipe.
//
// o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = 2^(s_ij - m_i), s_ij = q_i . k_j *
// log2(e) / sqrt(D) over the cached tokens, node i's ancestors and itself,
// in one pass over the keys with the running maximum m_i.
//
// A CTA of 256 threads takes its range of key tiles (64 keys) for R rows.
// Thread (ty, tx): rows ty + 16 i, keys tx + 16 j of the scores, then the same
// rows and channels 4 tx + 64 c of the output, so the softmax statistics of a
// row stay within 16 lanes and its accumulators see them without shared
// memory.  K and V have one buffer each, and each is refilled with the next
// tile while the other is in use; two CTAs per SM cover the rest.
#include "tree_common.cuh"

namespace dec {

namespace {

constexpr int kTreeKeys = 64;  // keys per tile: 4 pool blocks

template <int D, int R>
struct F32Smem {
  static constexpr int kPitch = D + 4;  // the 16 keys a half-warp reads fall into different banks
  static constexpr int kP = kTreeKeys + 4;
  static constexpr int kQ = 0, kK = kQ + R * kPitch, kV = kK + kTreeKeys * kPitch, kPr = kV + kTreeKeys * D;
  static constexpr int kBytes = (kPr + R * kP) * 4;
};

__device__ __forceinline__ void cp16(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int R>
__global__ void __launch_bounds__(256, D == 128 ? 2 : 3) k_tree_attend_f32(const __grid_constant__ TreeAttendArgs a) {
  // the plan is older than the kernels before this one: read before they are waited for
  const int here = tree_place();
  const TreeCut cut = a.m.cuts[here];
  const bool ok = tree_shape_ok(a.m, true);
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok) return;
  using SM = F32Smem<D, R>;
  constexpr int kRows = R / 16, kVec = D / 64 > 0 ? D / 64 : 1, kW = D >= 64 ? 4 : 2;  // channels: kVec groups of kW
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm + SM::kQ, *Ks = sm + SM::kK, *Vs = sm + SM::kV, *Ps = sm + SM::kPr;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int gs = a.d.gs, G = 1 << gs;
  TreeUnit u = tree_unit_first(a.m, cut);
  int tile = cut.tile;

  for (int left = cut.count; left > 0;) {
    const int t0 = tile, t1 = min(u.tiles, tile + left), end = u.ctx + u.nodes;
    const int32_t* table = a.m.tables + u.tab;
    auto load = [&](float* dst, int pitch, int t, int is_v) {
#pragma unroll
      for (int i = tid; i < kTreeKeys * (D / 4); i += 256) {
        const int r = i / (D / 4), c = i % (D / 4), key = t * kTreeKeys + r;
        const bool ok = key < end;
        int blk = ok ? __ldg(table + (key >> 4)) : 0;
#ifdef DEC_DEBUG
        if ((unsigned)blk >= (unsigned)a.d.n_blocks) {
          atomicOr(a.m.err, kErrBounds);
          blk = 0;
        }
#endif
        const float* src = reinterpret_cast<const float*>(a.kv) +
                           kv_offset(a.layer, blk, is_v, u.head, key & 15, a.d.n_blocks, a.d.Hkv, 16, D) + c * 4;
        cp16(dst + r * pitch + c * 4, src, ok);
      }
      cp_commit();
    };
    load(Ks, SM::kPitch, t0, 0);
    load(Vs, D, t0, 1);
    // this unit's queries (zeros past its last row)
    const int rows = min(R, u.nodes * G - u.row_tile * R);
    for (int i = tid; i < R * (D / 4); i += 256) {
      const int r = i / (D / 4), c = i % (D / 4), row = u.row_tile * R + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = tree_load4(a.q, a.q_type, (u.node0 + (row >> gs)) * a.ldq + (int64_t)(u.head * G + (row & (G - 1))) * D + c * 4);
      *reinterpret_cast<float4*>(Qs + r * SM::kPitch + c * 4) = v;
    }
    float m[kRows], l[kRows], o[kRows][kVec][kW];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < kVec; ++c)
#pragma unroll
        for (int e = 0; e < kW; ++e) o[i][c][e] = 0.f;
    }
    bool odd = false;  // a node's value of this unit is not finite
    for (int t = t0; t < t1; ++t) {
      cp_wait<1>();
      __syncthreads();  // K of this tile (and, first time, Q)
      float s[kRows][4];
#pragma unroll
      for (int i = 0; i < kRows; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll 2
      for (int d = 0; d < D; d += 4) {
        float4 q[kRows], k[4];
#pragma unroll
        for (int i = 0; i < kRows; ++i) q[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * SM::kPitch + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * SM::kPitch + d);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(q[i].x, k[j].x, s[i][j]);
            s[i][j] = fmaf(q[i].y, k[j].y, s[i][j]);
            s[i][j] = fmaf(q[i].z, k[j].z, s[i][j]);
            s[i][j] = fmaf(q[i].w, k[j].w, s[i][j]);
          }
      }
      __syncthreads();  // every thread is done with K
      if (t + 1 < t1) load(Ks, SM::kPitch, t + 1, 0);
      else cp_commit();
      const bool drafted = (t + 1) * kTreeKeys > u.ctx;  // some key of the tile is not a cached token
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = ty + 16 * i;
        const int node = u.node0 + min((u.row_tile * R + r) >> gs, u.nodes - 1);
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = t * kTreeKeys + tx + 16 * j - u.ctx;  // negative: a cached token
          s[i][j] *= a.scale_log2;
          if (drafted && n >= 0 && (n >= u.nodes || !tree_sees(a.m, node, n))) s[i][j] = -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m[i], mx), mu = mn == -INFINITY ? 0.f : mn;
        const float f = ex2(m[i] - mu);  // 0 for the first tile that a row sees anything of
        m[i] = mn;
        float ps = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = ex2(s[i][j] - mu);
          ps += p;
          Ps[r * SM::kP + tx + 16 * j] = p;
        }
        l[i] = fmaf(l[i], f, ps);  // this lane's keys; summed over the lanes at the end
#pragma unroll
        for (int c = 0; c < kVec; ++c)
#pragma unroll
          for (int e = 0; e < kW; ++e) o[i][c][e] *= f;
      }
      cp_wait<1>();
      __syncthreads();  // V of this tile and the weights
      if (drafted) {
        // a node's value that is not finite must not meet another branch's zero weights: zero it; its descendants get it
        // back at the unit's end
        bool found = false;
#pragma unroll 1
        for (int x = max(u.ctx - t * kTreeKeys, 0) * D + tid; x < kTreeKeys * D; x += 256)
          if (!isfinite(Vs[x])) {
            Vs[x] = 0.f;
            found = true;
          }
        odd |= __syncthreads_or(found);
      }
#pragma unroll 1
      for (int k0 = 0; k0 < kTreeKeys; k0 += 4) {
        float p[kRows][4];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * SM::kP + k0);
          p[i][0] = v.x;
          p[i][1] = v.y;
          p[i][2] = v.z;
          p[i][3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int c = 0; c < kVec; ++c) {
            float v[kW];
            const float* at = Vs + (k0 + k) * D + c * 64 + tx * kW;
            if constexpr (kW == 4) {
              const float4 w = *reinterpret_cast<const float4*>(at);
              v[0] = w.x;
              v[1] = w.y;
              v[2] = w.z;
              v[3] = w.w;
            } else {
              const float2 w = *reinterpret_cast<const float2*>(at);
              v[0] = w.x;
              v[1] = w.y;
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
              for (int e = 0; e < kW; ++e) o[i][c][e] = fmaf(p[i][k], v[e], o[i][c][e]);
          }
      }
      __syncthreads();  // every thread is done with V and the weights
      if (t + 1 < t1) load(Vs, D, t + 1, 1);
      else cp_commit();
    }
    cp_wait<0>();
    // the unit's rows: final, or this CTA's record of a shared unit
    const bool whole = t0 == 0 && t1 == u.tiles;
    float* rec = tree_record(a, here, t0 == 0);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
      const int r = ty + 16 * i, row = u.row_tile * R + r;
      if (r >= rows) continue;
      const int node = u.node0 + (row >> gs);
      if (odd) {  // rare: the values that were taken out, for the rows that see them
#pragma unroll 1
        for (int n = max(t0 * kTreeKeys - u.ctx, 0); n < min(t1 * kTreeKeys - u.ctx, u.nodes); ++n) {
          if (!tree_sees(a.m, node, n)) continue;
          const int p = u.ctx + n;
          const float* at = reinterpret_cast<const float*>(a.kv) +
                            kv_offset(a.layer, __ldg(table + (p >> 4)), 1, u.head, p & 15, a.d.n_blocks, a.d.Hkv, 16, D);
#pragma unroll
          for (int c = 0; c < kVec; ++c)
#pragma unroll
            for (int e = 0; e < kW; ++e) {
              const float v = at[c * 64 + tx * kW + e];
              if (!isfinite(v)) o[i][c][e] += v;
            }
        }
      }
      const bool zero = __ldg(a.m.pos + node) < 0 || l[i] == 0.f;
      const float f = whole ? 1.0f / l[i] : 1.f;
      const int64_t off = node * a.ldo + (int64_t)(u.head * G + (row & (G - 1))) * D;
#pragma unroll
      for (int c = 0; c < kVec; ++c) {
        const int d = c * 64 + tx * kW;
        float v[kW];
#pragma unroll
        for (int e = 0; e < kW; ++e) v[e] = whole && zero ? 0.f : o[i][c][e] * f;
        if constexpr (kW == 4) {
          const float4 w = make_float4(v[0], v[1], v[2], v[3]);
          if (whole) tree_store4(a.out, a.out_type, off + d, w);
          else *reinterpret_cast<float4*>(rec + r * D + d) = w;
        } else {
#pragma unroll
          for (int e = 0; e < kW; ++e) {
            if (whole) tree_store(a.out, a.out_type, off + d + e, v[e]);
            else rec[r * D + d + e] = v[e];
          }
        }
      }
      if (!whole && tx == 0) {
        rec[R * D + r] = m[i];
        rec[R * D + R + r] = l[i];
      }
    }
    left -= t1 - t0;
    tile = 0;
    if (left > 0) tree_unit_next(a.m, gs, R, a.d.Hkv, u);
  }
}

template <int D, int R>
cudaError_t one(const TreeAttendArgs& a, int ctas, cudaStream_t s) {
  static SmemOptIn opt;
  constexpr int smem = F32Smem<D, R>::kBytes;
  cudaError_t e = opt.ensure(k_tree_attend_f32<D, R>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_attend_f32<D, R>, ctas, 256, smem, s, a);
}

template <int D>
cudaError_t pick(const TreeAttendArgs& a, int ctas, cudaStream_t s) {
  return a.m.row_tile == 16 ? one<D, 16>(a, ctas, s) : one<D, 32>(a, ctas, s);
}

}  // namespace

cudaError_t launch_tree_attend_f32(const TreeAttendArgs& a, int ctas, cudaStream_t s) {
  switch (a.d.D) {
    case 32: return pick<32>(a, ctas, s);
    case 64: return pick<64>(a, ctas, s);
    case 128: return pick<128>(a, ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dec
