// kernels_tree_q8.cu - tree attention over a cache held in 8 bits, on the
// warp-level f16 tensor cores.
//
// o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = 2^(s_ij - m_i), s_ij = q_i . k_j *
// log2(e) / sqrt(D), with k_j = 2^a c_j and v_j = 2^b d_j, a and b the exponents
// of the pages that hold them.  The products run on the codes, which are exact
// in f16; 2^a goes into the scores' factor, b is added to the scores:
//   w_ij = 2^(s_ij + b - m_i),   O += w_ij d_j,   l += w_ij 2^-b.
// (Weights and reference go by the same rounded s_ij + b: with 2^b as a factor of
// p_ij, scores from 2^27 on, which have no place left for b, gave weights of 2^b.)
// The reference m_i is a running maximum of s_ij + b (raised when a row exceeds
// it by 2^8), so the rounded weights are at most 2^8 whatever the scales, and the
// largest at least 1; l holds in fp32 for scales of 2^-40 .. 2^40.
//
// The division of the work and the roundings are those of kernels_tree_f16.cu:
// a producer warp streams 64 keys (4 pool blocks, K and V, one TMA box per
// block) into a ring, warp w of four folds block w of every tile for 8 or 16
// rows.  Half the bytes a key leave half the time for it, so keys and channels
// take the 16 rows of the MMAs and the few query rows their 8 columns:
//   S^T = K Q^T, O^T += V^T P^T
// with half the MMAs of the other way round where 8 rows are enough (a decode
// step has 1 to 4), the queries in registers for a whole unit, and a maximum
// that is only formed when some weight would pass 2^8 (one vote a block).
//
// Codes to f16 without moving them between lanes: a dot product does not mind
// the order of its channels, so a lane's word of four codes, as it comes out of
// ldmatrix, is four channels in a row of one key, and the lane's queries the same
// four channels.  Values are read transposed in pairs of channels, a word holds
// two channels of two keys: its even bytes are an operand row of an even channel
// (rows 0 .. 7 of V^T's 16), its odd ones of an odd channel (rows 8 .. 15).
// Weights come as [key][row] and are needed as [row][key]: one 8 x 8 transpose
// (movmatrix) per 8 keys.
// i8: the byte, its sign flipped, under an exponent of 2^10 is 1024 + 128 + c in
// f16, one subtraction gives c: 5 instructions for four codes.
//
// 32 x 1 nodes over 1024-2048 keys, 16:8 heads x 128: 24.7 us, 102 MB at 4.1 TB/s;
// 32 x 1 over 6000 66 us, 6.0 TB/s (f16: 117 us).  From 1500 to 6000 keys a key's
// bytes go at 6.9 TB/s, so HBM bounds the long ones; some 9 us a call (the start,
// the ends of units, the second kernel) do not depend on the length.
#include "attn_fold.cuh"
#include "q8.cuh"
#include "tc_common.cuh"

namespace dec {

namespace {

constexpr int kQ8Keys = 64;  // keys per tile: 4 pool blocks
constexpr int kQ8Threads = 160;

template <int D, int R>
struct Q8Smem {
  static constexpr int kSlab = 16 * D;                         // K (or V) of one block
  static constexpr int kStage = 4 * 2 * kSlab;
  static constexpr int kCtas = D == 128 && R == 16 ? 2 : 3;    // per SM: with 16 rows of 128 channels a lane takes 168 registers, and spills 16 to 22 words at that
  static constexpr int kStages = D == 128 ? 4 : D == 64 ? 8 : 16;  // (two CTAs of 16 rows with six: 32 x 8 over 1500 36.0 us, with four 32.3)
  static constexpr int kQPitch = D * 2 + 16;                   // bytes; rows fall into different banks
  static constexpr int kQ = kStages * kStage;                  // the queries, at a unit's end the warps' outputs
  static constexpr int kRedPitch = 40;                         // floats of a row's 32 channels: rows fall into different banks
  static constexpr int kRed = 4 * R * kRedPitch * 4;
  static constexpr int kML = kQ + (R * kQPitch > kRed ? R * kQPitch : kRed);  // float [4][R] maxima, [4][R] sums
  static constexpr int kFac = kML + 2 * 4 * R * 4;       // float [R]: the rows' score factors
  static constexpr int kBar = kFac + R * 4;
  static constexpr int kBytes = kBar + 2 * kStages * 8 + 16;
  static_assert(kML % 16 == 0 && kBar % 8 == 0, "alignment");
};

// Byte offset of (row r, 16 channels from 16 c) in a block's K or V slab: rows of D bytes, swizzled as wide.
template <int D>
__device__ __forceinline__ int slab_at(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : D == 64 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) << 4);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Transpose of an 8 x 8 matrix of halves: a lane holds two of a row, before and after.
__device__ __forceinline__ uint32_t q8_transpose(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int R, int kKind>
__global__ void __launch_bounds__(kQ8Threads, Q8Smem<D, R>::kCtas) k_tree_attend_q8(const __grid_constant__ CUtensorMap tm,
                                                                  const __grid_constant__ TreeAttendArgs a) {
  using SM = Q8Smem<D, R>;
  constexpr int kN = R / 8, kS = SM::kStages;  // column tiles of 8 rows
  extern __shared__ __align__(1024) uint8_t dsm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(dsm + SM::kBar);
  uint64_t* empty = full + kS;
  int* flags = reinterpret_cast<int*>(empty + kS);  // [0] abort
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    flags[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the plan is older than the kernels before this one: read before they are waited for
  const int here = tree_place();
  const TreeCut cut = a.m.cuts[here];
  const bool ok_shape = tree_shape_ok(a.m, true);
  TreeUnit u = tree_unit_first(a.m, cut);
  int tile = cut.tile, k = 0;
  // pool block b of the current unit, if that is in front of block end
  auto entry = [&](int b, int end) {
    int blk = b < end ? __ldg(a.m.tables + u.tab + b) : 0;
#ifdef DEC_DEBUG
    if ((unsigned)blk >= (unsigned)a.d.n_blocks) {
      atomicOr(a.m.err, kErrBounds);
      blk = 0;
    }
#endif
    return blk;
  };
  auto blocks_to = [&](int t1) { return min((u.ctx + u.nodes + 15) >> 4, t1 * 4); };
  // a producer's lane: a block of the eight tiles from t on; a consumer's: warp w's block of the 32 tiles from t on
  auto entries = [&](int t, int t1) { return entry(warp == 4 ? t * 4 + lane : (t + lane) * 4 + warp, blocks_to(t1)); };
  int nxt = ok_shape && cut.count > 0 ? entries(tile, min(u.tiles, tile + cut.count)) : 0;
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
          tma_load_4d(dsm + slot * SM::kStage + lane * 2 * SM::kSlab, &tm, u.head * 16, a.layer * a.d.n_blocks + blk,
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
    const int key = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
    const int vkey = (lane & 7) + ((lane >> 3) & 1) * 8, vc = lane >> 4;
    bool alive = true;
    for (int left = cut.count; left > 0;) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), end = u.ctx + u.nodes;
      const int rows = min(R, u.nodes * G - u.row_tile * R);
      if (left < cut.count) nxt = entries(t0, t1);
      // the scales of this warp's blocks of 32 tiles, a lane each; the next ones' on their way while these are used
      auto scales_of = [&](int t, int blk) {
        float2 s = make_float2(1.f, 1.f);
        if ((t + lane) * 4 + warp < blocks_to(t1)) s = *reinterpret_cast<const float2*>(a.scales + q8_scale_at(a.d, a.layer, blk, u.head, 0));
        return make_float2(q8_two(q8_exp(s.x)), (float)q8_exp(s.y));
      };
      float2 sc = scales_of(t0, nxt), sc_next = sc;
      nxt = entries(t0 + 32, t1);
      auto put = [&](int r, int x, uint4 h) { *reinterpret_cast<uint4*>(Qs + r * SM::kQPitch + x * 16) = h; };
      constexpr int kLoaders = R * (D / 8) / 32 < 4 ? R * (D / 8) / 32 : 4;  // a warp reads 32 / (D / 8) rows at a time
      if (warp < kLoaders) tree_load_queries<D, R, kLoaders, 4>(a, u, u.row_tile * R, warp, fac, put);
      group_bar();
      // the lane's rows n * 8 + (lane >> 2) as operands, and n * 8 + 2 * (lane & 3), + 1 as columns of scores and outputs
      uint32_t q[kN][D / 16][2];
      float c[kN][2], m[kN][2], l[kN][2], o[kN][D / 16][4];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint2 x = *reinterpret_cast<const uint2*>(Qs + (n * 8 + (lane >> 2)) * SM::kQPitch + i * 32 + (lane & 3) * 8);
          q[n][i][0] = x.x;
          q[n][i][1] = x.y;
          o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          c[n][z] = fac[n * 8 + 2 * (lane & 3) + z];
          m[n][z] = -INFINITY;
          l[n][z] = 0.f;
        }
      }

      for (int t = t0; t < t1; ++t, ++k) {
        const int turn = (t - t0) & 31;
        if (turn == 0 && t > t0) {
          sc = sc_next;
          nxt = entries(t + 32, t1);
        }
        if (turn == 16 && t + 16 < t1) sc_next = scales_of(t + 16, nxt);
        const float sk = __shfl_sync(0xffffffffu, sc.x, turn), ev = __shfl_sync(0xffffffffu, sc.y, turn);
        const int slot = k % kS, key0 = t * kQ8Keys + warp * 16, nkeys = min(16, end - key0);
        const bool drafted = nkeys > 0 && key0 + nkeys > u.ctx;  // some key of the block is a node
        uint32_t sees[kN][2];  // this lane's columns, bit = key of the block; read ahead of the wait
        if (drafted) {
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int row = u.row_tile * R + n * 8 + 2 * (lane & 3) + z;
              sees[n][z] = tree_window(a.m, a.m.anc + (size_t)(u.node0 + min(row >> gs, u.nodes - 1)) * a.m.words, key0 - u.ctx);
            }
        }
        alive = __all_sync(0xffffffffu, alive && mbar_wait(&full[slot], (k / kS) & 1, abort_flag, a.m.err));
        if (alive && nkeys > 0) {
          const uint32_t kb = smem_u32(dsm) + slot * SM::kStage + warp * 2 * SM::kSlab, vb = kb + SM::kSlab;
          float s[kN][2][4];  // in two chains
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) s[n][z][0] = s[n][z][1] = s[n][z][2] = s[n][z][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t w[4];
            af_ldsm4(kb + slab_at<D>(key, kk * 2 + kc), w);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint32_t A[4];
              q8_halves<kKind, false>(w[z], A[0], A[2]);
              q8_halves<kKind, false>(w[2 + z], A[1], A[3]);
#pragma unroll
              for (int n = 0; n < kN; ++n) af_mma_f16(s[n][z], A, q[n][2 * kk + z][0], q[n][2 * kk + z][1]);
            }
          }
          // scores + ev of keys lane >> 2 and + 8: x[0], x[2] of the first column, x[1], x[3] of the second
          float x[kN][4];
          bool raise = false;
#pragma unroll
          for (int n = 0; n < kN; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[n][i] = fmaf(s[n][0][i] + s[n][1][i], fminf(c[n][i & 1] * sk, 3.40282347e38f), ev);
              if (drafted && !((sees[n][i & 1] >> ((lane >> 2) + (i >> 1) * 8)) & 1u)) x[n][i] = -INFINITY;
            }
            raise |= fmaxf(x[n][0], x[n][2]) - m[n][0] > 8.f || fmaxf(x[n][1], x[n][3]) - m[n][1] > 8.f;  // (m + 8 could round up to the next score)
          }
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                float mx = fmaxf(x[n][z], x[n][z + 2]);
#pragma unroll
                for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mn = fmaxf(m[n][z], mx);
                const float f = mn == m[n][z] ? 1.f : ex2(m[n][z] - mn);
                m[n][z] = mn;
                l[n][z] *= f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                  o[n][j][z] *= f;
                  o[n][j][z + 2] *= f;
                }
              }
          }
          const float out_of = q8_two(-(int)ev);
          uint32_t P[kN][2];
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              p[i] = ex2(x[n][i] - (m[n][i & 1] == -INFINITY ? 0.f : m[n][i & 1]));  // nothing seen so far: every weight is 0
              l[n][i & 1] = fmaf(p[i], out_of, l[n][i & 1]);
            }
            P[n][0] = q8_transpose(af_pack_half(p[0], p[1]));
            P[n][1] = q8_transpose(af_pack_half(p[2], p[3]));
          }
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t w[4];
            af_ldsm4t(vb + slab_at<D>(vkey, j * 2 + vc), w);
            if (kKind == kTreeE4m3 && drafted) {  // rows of no node hold anything, and 0 times NaN is NaN
#pragma unroll
              for (int z = 0; z < 4; ++z) w[z] = e4m3_numbers(w[z]);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {  // 16 channels: keys 0 .. 7 and 8 .. 15
              uint32_t A[4];
              q8_halves<kKind, true>(w[2 * z], A[0], A[1]);
              q8_halves<kKind, true>(w[2 * z + 1], A[2], A[3]);
#pragma unroll
              for (int n = 0; n < kN; ++n) af_mma_f16(o[n][2 * j + z], A, P[n][0], P[n][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
      }
      // ---- the unit's end: the four warps' states in warp order ----
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[n][z] += __shfl_xor_sync(0xffffffffu, l[n][z], d);
          if (lane < 4) {
            const int r = n * 8 + 2 * lane + z;
            ml[warp * R + r] = m[n][z];
            ml[(4 + warp) * R + r] = l[n][z];
          }
        }
      group_bar();
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // this warp's factor to the common maximum
          const int r = n * 8 + 2 * (lane & 3) + z;
          const float M = fmaxf(fmaxf(ml[r], ml[R + r]), fmaxf(ml[2 * R + r], ml[3 * R + r]));
          const float f = ex2(m[n][z] - (M == -INFINITY ? 0.f : M));  // 0 where the row saw nothing
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[n][j][z] *= f;
            o[n][j][z + 2] *= f;
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
          part[R * D + r] = M;
          part[R * D + R + r] = L;
        }
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {  // 32 channels at a time
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int z = 0; z < 2; ++z)  // channels 2 (lane >> 2), + 1 of 16
              *reinterpret_cast<float2*>(red + (warp * R + n * 8 + 2 * (lane & 3) + z) * SM::kRedPitch + i * 16 + 2 * (lane >> 2)) =
                  make_float2(o[n][2 * j + i][z], o[n][2 * j + i][z + 2]);
        group_bar();
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
          if (!whole) {
            *reinterpret_cast<float4*>(part + r * D + j * 32 + x) = v;
          } else {
            const int row = u.row_tile * R + r;
            const float f = fac[r];
            tree_store4(a.out, a.out_type, (u.node0 + (row >> gs)) * a.ldo + (int64_t)(u.head * G + (row & (G - 1))) * D + j * 32 + x,
                        f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
          }
        }
        group_bar();
      }
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

template <int D, int R, int kKind>
cudaError_t one(const TreeAttendArgs& a, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  static SmemOptIn opt;
  constexpr int smem = Q8Smem<D, R>::kBytes;
  static_assert(smem <= 76 * 1024, "three CTAs per SM");
  cudaError_t e = opt.ensure(k_tree_attend_q8<D, R, kKind>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_attend_q8<D, R, kKind>, ctas, kQ8Threads, smem, s, *tm, a);
}
template <int D>
cudaError_t kinds(const TreeAttendArgs& a, int kv_type, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  if (a.m.row_tile == 8) return kv_type == kTreeI8 ? one<D, 8, kTreeI8>(a, tm, ctas, s) : one<D, 8, kTreeE4m3>(a, tm, ctas, s);
  return kv_type == kTreeI8 ? one<D, 16, kTreeI8>(a, tm, ctas, s) : one<D, 16, kTreeE4m3>(a, tm, ctas, s);
}

}  // namespace

cudaError_t launch_tree_attend_q8(const TreeAttendArgs& a, int kv_type, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  switch (a.d.D) {
    case 32: return kinds<32>(a, kv_type, tm, ctas, s);
    case 64: return kinds<64>(a, kv_type, tm, ctas, s);
    case 128: return kinds<128>(a, kv_type, tm, ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dec
