// kernels_tree_f16.cu - tree attention over an f16 cache (the serving modes)
// on the warp-level f16 tensor cores.
//
// o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = 2^(s_ij - m_i), s_ij = q_i . k_j *
// log2(e) / sqrt(D) over the cached tokens, node i's ancestors and itself.
//
// A CTA takes a contiguous range of key tiles.  A producer warp streams each
// tile (64 keys: 4 pool blocks, K and V, one 5-D TMA box per block) into a
// ring; warp w of four folds block w of every tile for all R rows, so the
// warps meet only at a unit's end: S = Q K^T by m16n8k16, the softmax in
// fp32, O += P V with the accumulator in registers.  The running maximum is
// raised (and O rescaled) only when a row's scores exceed it by 2^8, which
// leaves the result exact: numerator and denominator use the same maximum.
//
// Rounded to f16: the queries, each row scaled by a power of two to [1, 2)
// first so that no magnitude overflows (off by at most 2^-11 of the row's
// largest channel; the cached keys are f16 already), and the weights P (2^-11
// relative each, or 2^-25 where that is more; they are at most 2^8 and the
// row's largest at least 1).  Statistics and accumulators are fp32.
#include "attn_fold.cuh"
#include "tc_common.cuh"
#include "tree_common.cuh"

namespace dec {

namespace {

constexpr int kTreeKeys = 64;  // keys per tile: 4 pool blocks

template <int D, int R>
struct F16Smem {
  static constexpr int kSlab = 16 * D * 2;                     // K (or V) of one block
  static constexpr int kStage = 4 * 2 * kSlab;
  static constexpr int kStages = D == 128 ? 3 : D == 64 ? 6 : 8;
  static constexpr int kQPitch = D * 2 + 16;                   // bytes; rows fall into different banks
  static constexpr int kQ = kStages * kStage;                  // the queries, at a unit's end the warps' outputs
  static constexpr int kRedPitch = 40;                         // floats of a row's 32 channels: rows fall into different banks
  static constexpr int kRed = 4 * R * kRedPitch * 4;
  static constexpr int kML = kQ + (R * kQPitch > kRed ? R * kQPitch : kRed);  // float [4][R] maxima, [4][R] sums
  static constexpr int kFac = kML + 2 * 4 * R * 4;             // float [R]: the rows' score factors
  static constexpr int kBar = kFac + R * 4;
  static constexpr int kBytes = kBar + 2 * kStages * 8 + 16;
  static_assert(kML % 16 == 0 && kBar % 8 == 0, "alignment");
};

// Byte offset of (row r, channels d .. d+7) in a block's K or V slab.
template <int D>
__device__ __forceinline__ int slab_at(int r, int d) {
  if constexpr (D >= 64) return (d >> 6) * 2048 + r * 128 + ((((d >> 3) & 7) ^ (r & 7)) << 4);
  else return r * 64 + (((d >> 3) ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %2, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

constexpr int kF16Threads = 160;

template <int D, int R>
__global__ void __launch_bounds__(kF16Threads, 2) k_tree_attend_f16(const __grid_constant__ CUtensorMap tm,
                                                                    const __grid_constant__ TreeAttendArgs a) {
  using SM = F16Smem<D, R>;
  constexpr int MT = R / 16, kS = SM::kStages;
  extern __shared__ __align__(1024) uint8_t dsm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(dsm + SM::kBar);
  uint64_t* empty = full + kS;
  int* flags = reinterpret_cast<int*>(empty + kS);  // [0] abort, [1] a node's value of this unit is not finite
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    flags[0] = flags[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the plan is older than the kernels before this one: read before they are waited for
  const int here = tree_place();
  const TreeCut cut = a.m.cuts[here];
  const bool ok_shape = tree_shape_ok(a.m, true);
  TreeUnit u = tree_unit_first(a.m, cut);
  int tile = cut.tile, k = 0;
  // a lane's block of the eight tiles from t on, of the current unit up to tile t1
  auto entries = [&](int t, int t1) {
    const int b = t * 4 + lane;
    int blk = b < (u.ctx + u.nodes + 15) >> 4 && b < t1 * 4 ? __ldg(a.m.tables + u.tab + b) : 0;
#ifdef DEC_DEBUG
    if ((unsigned)blk >= (unsigned)a.d.n_blocks) {
      atomicOr(a.m.err, kErrBounds);
      blk = 0;
    }
#endif
    return blk;
  };
  int nxt = warp == 4 && ok_shape && cut.count > 0 ? entries(tile, min(u.tiles, tile + cut.count)) : 0;
  __syncthreads();
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok_shape) return;
  volatile int* abort_flag = flags;
  const int gs = a.d.gs, G = 1 << gs;

  if (warp == 4) {
    // ---- producer: lanes 0..3 copy one block each; table entries come 8 tiles at a time ----
    for (int left = cut.count; left > 0;) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), blocks = (u.ctx + u.nodes + 15) >> 4;
      if (left < cut.count) nxt = entries(t0, t1);  // the first unit's are there
      int cur = 0;
      for (int t = t0; t < t1; ++t, ++k) {
        if (((t - t0) & 7) == 0) {
          cur = nxt;
          nxt = entries(t + 8, t1);
        }
        const int blk = __shfl_sync(0xffffffffu, cur, (((t - t0) & 7) << 2) + (lane & 3));
        const int slot = k % kS;
        bool ok = true;
        if (lane == 0 && k >= kS) ok = mbar_wait(&empty[slot], ((k / kS) - 1) & 1, abort_flag, a.m.err);
        if (!__shfl_sync(0xffffffffu, (int)ok, 0)) goto produced;
        if (lane == 0) mbar_expect_tx(&full[slot], min(4, blocks - t * 4) * 2 * SM::kSlab);
        __syncwarp();
        if (lane < 4 && t * 4 + lane < blocks)
          tma_load_5d(dsm + slot * SM::kStage + lane * 2 * SM::kSlab, &tm, u.head * 16, a.layer * a.d.n_blocks + blk,
                      &full[slot]);
        __syncwarp();
      }
      left -= t1 - t0;
      tile = 0;
      if (left > 0) tree_unit_next(a.m, gs, R, a.d.Hkv, u);
    }
  produced:;
  } else {
    // ---- consumers: warp w folds block w of every tile ----
    uint8_t* Qs = dsm + SM::kQ;
    float* red = reinterpret_cast<float*>(dsm + SM::kQ);
    float* ml = reinterpret_cast<float*>(dsm + SM::kML);
    float* fac = reinterpret_cast<float*>(dsm + SM::kFac);
    auto group_bar = []() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    const int key = (lane & 7) + ((lane >> 4) << 3), doff = ((lane >> 3) & 1) * 8;
    const int vkey = (lane & 7) + ((lane >> 3) & 1) * 8, vd = (lane >> 4) * 8;
    bool alive = true;
    for (int left = cut.count; left > 0;) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), end = u.ctx + u.nodes;
      const int rows = min(R, u.nodes * G - u.row_tile * R);
      if constexpr (R / 4 >= 32 / (D / 8)) {
        tree_load_queries<D, R, 4, 4>(a, u, u.row_tile * R, warp, fac, [&](int r, int x, uint4 h) { *reinterpret_cast<uint4*>(Qs + r * SM::kQPitch + x * 16) = h; });
      } else if (warp < 2) {  // D = 32, R = 16: a warp reads eight rows at a time
        tree_load_queries<D, R, 2, 4>(a, u, u.row_tile * R, warp, fac, [&](int r, int x, uint4 h) { *reinterpret_cast<uint4*>(Qs + r * SM::kQPitch + x * 16) = h; });
      }
      group_bar();
      const uint32_t qb = smem_u32(Qs) + (lane & 15) * SM::kQPitch + (lane >> 4) * 16;
      float c[2 * MT], m[2 * MT], l[2 * MT], o[MT][D / 8][4];
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        c[i] = fac[(i >> 1) * 16 + (i & 1) * 8 + (lane >> 2)];
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;

      for (int t = t0; t < t1; ++t, ++k) {
        const int slot = k % kS, key0 = t * kTreeKeys + warp * 16, nkeys = min(16, end - key0);
        const bool drafted = nkeys > 0 && key0 + nkeys > u.ctx;  // some key of the block is a node
        uint32_t sees[2 * MT];  // this lane's rows, bit = key of the block; read ahead of the wait
        if (drafted) {
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            const int row = u.row_tile * R + (i >> 1) * 16 + (i & 1) * 8 + (lane >> 2);
            sees[i] = tree_window(a.m, a.m.anc + (size_t)(u.node0 + min(row >> gs, u.nodes - 1)) * a.m.words, key0 - u.ctx);
          }
        }
        alive = __all_sync(0xffffffffu, alive && mbar_wait(&full[slot], (k / kS) & 1, abort_flag, a.m.err));
        if (alive && nkeys > 0) {
          uint8_t* Kb = dsm + slot * SM::kStage + warp * 2 * SM::kSlab;
          uint8_t* Vb = Kb + SM::kSlab;
          const uint32_t kb = smem_u32(Kb), vb = smem_u32(Vb);
          float s[MT][2][4];
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t B[4];
            af_ldsm4(kb + slab_at<D>(key, kk * 16 + doff), B);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              uint32_t A[4];
              af_ldsm4(qb + i * 16 * SM::kQPitch + kk * 32, A);
              af_mma_f16(s[i][0], A, B[0], B[1]);
              af_mma_f16(s[i][1], A, B[2], B[3]);
            }
          }
          float mx[2 * MT];
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            float(&x)[2][4] = s[i >> 1];
            const int e = (i & 1) * 2;
            mx[i] = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              x[n][e] *= c[i];
              x[n][e + 1] *= c[i];
            }
            if (drafted) {
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int z = 0; z < 2; ++z)
                  if (!((sees[i] >> (n * 8 + 2 * (lane & 3) + z)) & 1u)) x[n][e + z] = -INFINITY;
            }
            mx[i] = fmaxf(fmaxf(x[0][e], x[0][e + 1]), fmaxf(x[1][e], x[1][e + 1]));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
          }
          bool raise = false;
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) raise |= mx[i] > m[i] + 8.f;
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
              const float mn = fmaxf(m[i], mx[i]);
              const float f = mn == m[i] ? 1.f : ex2(m[i] - mn);
              m[i] = mn;
              l[i] *= f;
#pragma unroll
              for (int j = 0; j < D / 8; ++j) {
                o[i >> 1][j][(i & 1) * 2] *= f;
                o[i >> 1][j][(i & 1) * 2 + 1] *= f;
              }
            }
          }
          uint32_t P[MT][4];
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            float(&x)[2][4] = s[i >> 1];
            const int e = (i & 1) * 2;
            const float mu = m[i] == -INFINITY ? 0.f : m[i];  // nothing seen so far: every weight is 0
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float p0 = ex2(x[n][e] - mu), p1 = ex2(x[n][e + 1] - mu);
              l[i] += p0 + p1;
              P[i >> 1][2 * n + (i & 1)] = af_pack_half(p0, p1);
            }
          }
          if (drafted) {
            // value rows past the end hold anything: zero them; a node's value that is not finite must not meet
            // another branch's zero weights: zero it too, its descendants get it back at the unit's end
            bool odd = false, changed = false;
#pragma unroll 4
            for (int i = max(u.ctx - key0, 0) * (D / 8) + lane; i < 16 * (D / 8); i += 32) {
              const int r = i / (D / 8);
              uint4* p = reinterpret_cast<uint4*>(Vb + slab_at<D>(r, (i % (D / 8)) * 8));
              uint4 x = *p;
              uint32_t* w = reinterpret_cast<uint32_t*>(&x);
              if (r < nkeys ? tree_not_finite(x) : (w[0] | w[1] | w[2] | w[3])) {
#pragma unroll
                for (int z = 0; z < 4; ++z) w[z] = r < nkeys ? tree_finite_or_0(w[z]) : 0u;
                *p = x;
                odd |= r < nkeys;
                changed = true;
              }
            }
            if (__any_sync(0xffffffffu, changed)) {
              if (__any_sync(0xffffffffu, odd) && lane == 0) flags[1] = 1;
              // the slot is refilled by the async proxy later: order these stores before it
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            }
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t B[4];
            af_ldsm4t(vb + slab_at<D>(vkey, j * 16 + vd), B);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              af_mma_f16(o[i][2 * j], P[i], B[0], B[1]);
              af_mma_f16(o[i][2 * j + 1], P[i], B[2], B[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
      }
      // ---- the unit's end: the four warps' states in warp order ----
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if ((lane & 3) == 0) {
          const int r = (i >> 1) * 16 + (i & 1) * 8 + (lane >> 2);
          ml[warp * R + r] = m[i];
          ml[(4 + warp) * R + r] = l[i];
        }
      }
      group_bar();
      const bool odd = flags[1] != 0;
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {  // this warp's factor to the common maximum
        const int r = (i >> 1) * 16 + (i & 1) * 8 + (lane >> 2);
        const float M = fmaxf(fmaxf(ml[r], ml[R + r]), fmaxf(ml[2 * R + r], ml[3 * R + r]));
        const float f = ex2(m[i] - (M == -INFINITY ? 0.f : M));  // 0 where the row saw nothing
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[i >> 1][j][(i & 1) * 2] *= f;
          o[i >> 1][j][(i & 1) * 2 + 1] *= f;
        }
      }
      // the rows are final here, or this CTA's part of a shared unit: a record
      const bool whole = t0 == 0 && t1 == u.tiles;
      float* part = tree_record(a, here, t0 == 0);
      if (threadIdx.x < rows) {
        const int r = threadIdx.x;
        const float M = fmaxf(fmaxf(ml[r], ml[R + r]), fmaxf(ml[2 * R + r], ml[3 * R + r]));
        // no maximum: the row saw nothing (its sums are 0), or every score of it was NaN (so is a sum, and the output)
        const float mu = M == -INFINITY ? 0.f : M;
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) L += ml[(4 + w) * R + r] * ex2(ml[w * R + r] - mu);
        if (whole) {
          const bool zero = L == 0.f || __ldg(a.m.pos + u.node0 + ((u.row_tile * R + r) >> gs)) < 0;
          fac[r] = zero ? 0.f : 1.0f / L;
        } else {
          fac[r] = 1.f;
          part[R * D + r] = M;
          part[R * D + R + r] = L;
        }
      }
      auto out_at = [&](int r) {  // element of the output's first channel of row r
        const int row = u.row_tile * R + r;
        return (u.node0 + (row >> gs)) * a.ldo + (int64_t)(u.head * G + (row & (G - 1))) * D;
      };
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {  // 32 channels at a time
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z)
              *reinterpret_cast<float2*>(red + (warp * R + i * 16 + z * 8 + (lane >> 2)) * SM::kRedPitch + n * 8 + 2 * (lane & 3)) =
                  make_float2(o[i][4 * j + n][2 * z], o[i][4 * j + n][2 * z + 1]);
        group_bar();
#pragma unroll 1
        for (int i = threadIdx.x; i < rows * 8; i += 128) {
          const int r = i >> 3, x = (i & 7) * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(red + (w * R + r) * SM::kRedPitch + x);
            v.x += y.x;
            v.y += y.y;
            v.z += y.z;
            v.w += y.w;
          }
          const float f = fac[r];
          if (!whole) *reinterpret_cast<float4*>(part + r * D + j * 32 + x) = v;
          else tree_store4(a.out, a.out_type, out_at(r) + j * 32 + x, f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        }
        group_bar();
      }
      if (odd) {  // rare: the values that were taken out, for the rows that see them
        const int32_t* table = a.m.tables + u.tab;
        const int j0 = max(t0 * kTreeKeys - u.ctx, 0), j1 = min(t1 * kTreeKeys - u.ctx, u.nodes);
#pragma unroll 1
        for (int i = threadIdx.x; i < rows * D; i += 128) {
          const int r = i / D, node = u.node0 + ((u.row_tile * R + r) >> gs);
          if (fac[r] == 0.f) continue;  // padding, or nothing seen
#pragma unroll 1
          for (int n = j0; n < j1; ++n) {
            if (!tree_sees(a.m, node, n)) continue;
            const int p = u.ctx + n;
            const float z = __half2float(reinterpret_cast<const __half*>(
                a.kv)[kv_offset(a.layer, __ldg(table + (p >> 4)), 1, u.head, p & 15, a.d.n_blocks, a.d.Hkv, 16, D) + i % D]);
            if (isfinite(z)) continue;
            if (whole) tree_store(a.out, a.out_type, out_at(r) + i % D, tree_load(a.out, a.out_type, out_at(r) + i % D) + z);
            else part[i] += z;
          }
        }
        group_bar();
      }
      if (threadIdx.x == 0) flags[1] = 0;
      group_bar();  // the statistics and the flag are free again
      left -= t1 - t0;
      tile = 0;
      if (left > 0) tree_unit_next(a.m, gs, R, a.d.Hkv, u);
    }
  }
  __syncthreads();
  // after an abort, let the copies still in flight land before the CTA exits
  if (warp == 4 && lane == 0 && *abort_flag) {
    const uint64_t w0 = global_ns();
    for (int i = k > kS ? k - kS : 0; i < k; ++i)
      while (!mbar_try(&full[i % kS], (i / kS) & 1) && global_ns() - w0 < kWaitLimitNs) {
      }
  }
}

template <int D, int R>
cudaError_t one(const TreeAttendArgs& a, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  static SmemOptIn opt;
  constexpr int smem = F16Smem<D, R>::kBytes;
  static_assert(smem <= 115712, "two CTAs per SM");
  cudaError_t e = opt.ensure(k_tree_attend_f16<D, R>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_attend_f16<D, R>, ctas, kF16Threads, smem, s, *tm, a);
}

}  // namespace

cudaError_t launch_tree_attend_f16(const TreeAttendArgs& a, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  switch (a.d.D) {
    case 32: return a.m.row_tile == 16 ? one<32, 16>(a, tm, ctas, s) : one<32, 32>(a, tm, ctas, s);
    case 64: return one<64, 16>(a, tm, ctas, s);
    case 128: return one<128, 16>(a, tm, ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dec
