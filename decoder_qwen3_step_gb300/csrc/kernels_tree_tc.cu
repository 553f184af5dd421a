// kernels_tree_tc.cu - tree attention over an f16 cache for wide trees, on the
// 5th-generation tensor cores (tcgen05, accumulators in TMEM).
//
// The same formula as kernels_tree_f16.cu with 128 rows (nodes x query heads
// of one KV head) and 128 keys per step:
//   warp 0      TMA producer: K and V tiles as 64-channel panels of 128 keys in
//               128-byte swizzled rows (one box per block and panel)
//   warp 1      issues S = Q K^T (both operands K-major in shared memory) and
//               O += P V (P from TMEM, V as a channel-major operand: its
//               panels are read transposed by the MMA itself)
//   warps 2..5  softmax: thread = row = TMEM lane.  S is read from TMEM, the
//               weights go back as f16 over the first half of the S columns,
//               so a row's maximum and sum never leave their thread
// S (128 columns) and O (D columns) fill half of TMEM: two CTAs per SM, and one
// CTA's softmax runs under the other's MMAs.  O is rescaled in TMEM only when
// a row's scores exceed its maximum by 2^8 (exact: numerator and denominator
// share the maximum).  Roundings as in kernels_tree_f16.cu.
#include "attn_fold.cuh"
#include "tc_common.cuh"
#include "tree_common.cuh"

namespace dec {

namespace {

constexpr int kTR = 128, kTK = 128;  // rows and keys of a step
constexpr int kTcTreeThreads = 192;
constexpr uint32_t kTmemCols = 256;  // S: columns 0..127, O: 128..128+D-1

template <int D>
struct TcSmem {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = kTK * 128;            // bytes of 64 channels of 128 keys (or rows)
  static constexpr int kTile = kPanels * kPanel;
  static constexpr int kStages = D == 128 ? 1 : 2;
  static constexpr int kQ = 0, kK = kTile, kV = kK + kStages * kTile, kFac = kV + kStages * kTile;
  static constexpr int kBar = kFac + kTR * 4;
  // barriers: K full, K empty, V full, V empty [stages]; Q full, S full, P full, O full, MMA done
  static constexpr int kBars = 4 * kStages + 5;
  static constexpr int kBytes = kBar + kBars * 8 + 32;
};

__device__ __forceinline__ void tma_box_5d(void* dst, const CUtensorMap* map, int y, int half, int is_v, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(y), "r"(half), "r"(is_v), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// D (TMEM) += A (TMEM, f16 pairs per column) B (shared memory)
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// Instruction descriptor, kind::f16: f16 operands, fp32 accumulator; bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// MN-major operand, 128-byte swizzle: 64-element atoms `panel` bytes apart, groups of 8 along K 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t panel) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

#define TREE_R32(v)                                                                                                 \
  "r"((v)[0]), "r"((v)[1]), "r"((v)[2]), "r"((v)[3]), "r"((v)[4]), "r"((v)[5]), "r"((v)[6]), "r"((v)[7]),           \
      "r"((v)[8]), "r"((v)[9]), "r"((v)[10]), "r"((v)[11]), "r"((v)[12]), "r"((v)[13]), "r"((v)[14]), "r"((v)[15])
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      TREE_R32(v)
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kTcTreeThreads, 2) k_tree_attend_tc(const __grid_constant__ CUtensorMap tm,
                                                                      const __grid_constant__ TreeAttendArgs a) {
  using SM = TcSmem<D>;
  constexpr int kS = SM::kStages;
  extern __shared__ __align__(1024) uint8_t dsm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsm + SM::kBar);
  uint64_t *kfull = bars, *kempty = bars + kS, *vfull = bars + 2 * kS, *vempty = bars + 3 * kS;
  uint64_t *qfull = bars + 4 * kS, *sfull = qfull + 1, *pfull = qfull + 2, *ofull = qfull + 3, *mma_done = qfull + 4;
  int* flags = reinterpret_cast<int*>(bars + SM::kBars);  // [0] abort, [1] odd values, [2] TMEM base, [3] tiles copied
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 1);
    }
    mbar_init(qfull, 128);
    mbar_init(sfull, 1);
    mbar_init(pfull, 128);
    mbar_init(ofull, 1);
    mbar_init(mma_done, 1);
    flags[0] = flags[1] = flags[3] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait_prev();
  pdl_launch_next();
  if (!tree_shape_ok(a.m, true)) return;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(flags + 2)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(flags + 2);
  volatile int* abort_flag = flags;
  const int G = a.d.H / a.d.Hkv;
  const TreeCut cut = a.m.cuts[blockIdx.x];
  TreeUnit u{cut.seq, cut.head, cut.row_tile, 0, 0, 0, 0, 0};
  if (cut.count > 0) tree_unit_load(a.m, G, kTR, u);
  int tile = cut.tile, k = 0;  // k: tiles so far, over all units

  if (warp == 0) {
    // ---- producer: lane = (panel, block) for K, then for V ----
    for (int left = cut.count; left > 0;) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), blocks = (u.ctx + u.nodes + 15) >> 4;
      const int32_t* table = a.m.tables + __ldg(a.m.tab_start + u.seq);
      auto entry = [&](int t) {
        const int b = t * 8 + (lane & 7);
        int blk = b < blocks && t < t1 ? __ldg(table + b) : 0;
#ifdef DEC_DEBUG
        if ((unsigned)blk >= (unsigned)a.d.n_blocks) {
          atomicOr(a.m.err, kErrBounds);
          blk = 0;
        }
#endif
        return blk;
      };
      int nxt = entry(t0);
      for (int t = t0; t < t1; ++t, ++k) {
        const int slot = k % kS, here = min(8, blocks - t * 8), blk = nxt;
        nxt = entry(t + 1);
        const uint32_t bytes = here * SM::kPanels * 2048;
        const int z = a.layer * a.d.n_blocks + blk, panel = lane >> 3;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
          uint64_t* full = is_v ? &vfull[slot] : &kfull[slot];
          uint64_t* empty = is_v ? &vempty[slot] : &kempty[slot];
          bool ok = true;
          if (lane == 0 && k >= kS) ok = mbar_wait(empty, ((k / kS) - 1) & 1, abort_flag, a.m.err);
          if (!__shfl_sync(0xffffffffu, (int)ok, 0)) goto produced;
          if (lane == 0) {
            mbar_expect_tx(full, bytes);
            flags[3] = 2 * k + 1 + is_v;
          }
          __syncwarp();
          if (panel < SM::kPanels && (lane & 7) < here)
            tma_box_5d(dsm + (is_v ? SM::kV : SM::kK) + slot * SM::kTile + panel * SM::kPanel + (lane & 7) * 2048, &tm,
                       u.head * 16, panel, is_v, z, full);
          __syncwarp();
        }
      }
      left -= t1 - t0;
      tile = 0;
      if (left > 0) tree_unit_next(a.m, G, kTR, a.d.Hkv, u);
    }
  produced:;
  } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f16(kTR, kTK, false), id_o = idesc_f16(kTR, D, true);
      const uint32_t qa = smem_u32(dsm + SM::kQ);
      int n_unit = 0;
      for (int left = cut.count; left > 0; ++n_unit) {
        const int t0 = tile, t1 = min(u.tiles, tile + left);
        if (!mbar_wait(qfull, n_unit & 1, abort_flag, a.m.err)) goto issued;
        for (int t = t0; t < t1; ++t, ++k) {
          const int slot = k % kS;
          if (!mbar_wait(&kfull[slot], (k / kS) & 1, abort_flag, a.m.err)) goto issued;
          tc_fence_after();
          const uint32_t ka = smem_u32(dsm + SM::kK + slot * SM::kTile), va = smem_u32(dsm + SM::kV + slot * SM::kTile);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = (i >> 2) * SM::kPanel + (i & 3) * 32;
            tc_mma(tmem, sw128_desc(qa + off), sw128_desc(ka + off), id_s, i != 0);
          }
          tc_commit(&kempty[slot]);
          tc_commit(sfull);
          if (!mbar_wait(&vfull[slot], (k / kS) & 1, abort_flag, a.m.err)) goto issued;
          if (!mbar_wait(pfull, k & 1, abort_flag, a.m.err)) goto issued;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kTK / 16; ++i)
            tc_mma_ts(tmem + 128, tmem + i * 8, sw128_mn_desc(va + i * 2048, SM::kPanel), id_o, t != t0 || i != 0);
          tc_commit(&vempty[slot]);
        }
        tc_commit(ofull);
        left -= t1 - t0;
        tile = 0;
        if (left > 0) tree_unit_next(a.m, G, kTR, a.d.Hkv, u);
      }
    issued:
      tc_commit(mma_done);
    }
    __syncwarp();
  } else {
    // ---- softmax: thread = row ----
    const int r = (warp & 3) * 32 + lane, st = threadIdx.x - 64;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float* fac = reinterpret_cast<float*>(dsm + SM::kFac);
    auto group_bar = []() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    int n_unit = 0;
    bool alive = true;
    for (int left = cut.count; left > 0; ++n_unit) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), end = u.ctx + u.nodes;
      const int rows = min(kTR, u.nodes * G - u.row_tile * kTR);
      tree_load_queries<D, kTR, 4>(a, u, G, warp - 2, fac, [&](int q, int x, uint2 h) {
        *reinterpret_cast<uint2*>(dsm + SM::kQ + (x >> 4) * SM::kPanel + q * 128 + ((((x & 15) >> 1) ^ (q & 7)) << 4) +
                                  (x & 1) * 8) = h;
      });
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(qfull);
      group_bar();
      const float c = fac[r];
      const int node = u.node0 + min((u.row_tile * kTR + r) / G, u.nodes - 1);
      const uint32_t* anc = a.m.anc + (size_t)node * a.m.words;
      float m = -INFINITY, l = 0.f;
      for (int t = t0; t < t1; ++t, ++k) {
        alive = __all_sync(0xffffffffu, alive && mbar_wait(sfull, k & 1, abort_flag, a.m.err));
        if (alive) {
          tc_fence_after();
          const int key0 = t * kTK;
          const bool drafted = key0 + kTK > u.ctx;
          // which of the 32 keys of column chunk j this row sees
          auto sees = [&](int j) -> uint32_t {
            const int b = key0 + j * 32 - u.ctx;  // node number of the chunk's first key; negative: cached tokens
            if (b <= -32) return 0xffffffffu;
            if (b < 0) return (__ldg(anc) << -b) | ((1u << -b) - 1u);
            const int w = b >> 5;
            const uint32_t lo = w < a.m.words ? __ldg(anc + w) : 0u, hi = w + 1 < a.m.words ? __ldg(anc + w + 1) : 0u;
            return __funnelshift_r(lo, hi, b & 31);
          };
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t s[32];
            tc_ld32(trow + j * 32, s);
            if (drafted) {
              const uint32_t vis = sees(j);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((vis >> i) & 1u) mx = fmaxf(mx, __uint_as_float(s[i]));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(s[i]));
            }
          }
          mx *= c;
          if (__any_sync(0xffffffffu, mx > m + 8.f)) {
            const float mn = fmaxf(m, mx), f = mn == m ? 1.f : ex2(m - mn);
            m = mn;
            l *= f;
            if (t > t0) {  // the MMAs of the tiles before have run (S of this one was issued behind them)
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {
                uint32_t o[32];
                tc_ld32(trow + 128 + j * 32, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tc_st16(trow + 128 + j * 32, o);
                tc_st16(trow + 128 + j * 32 + 16, o + 16);
              }
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
          // s c - m in one rounding while that is small against the weights' own (2^-12 at 2^12); far out the product is
          // rounded as the maximum was, or the largest score would miss it by its own last place
          const bool plain = !drafted && !__any_sync(0xffffffffu, !(fabsf(mu) <= 4096.f));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t s[32], p[16];
            tc_ld32(trow + j * 32, s);
            if (plain) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(ex2(fmaf(__uint_as_float(s[i]), c, -mu)));
            } else {
              const uint32_t vis = drafted ? sees(j) : 0xffffffffu;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = ex2(__fadd_rn(__fmul_rn(__uint_as_float(s[i]), c), -mu));
                s[i] = (vis >> i) & 1u ? __float_as_uint(x) : 0u;
              }
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float x = __uint_as_float(s[i]), y = __uint_as_float(s[i + 1]);
              l4[i & 2] += x;
              l4[(i & 2) + 1] += y;
              const __half2 h = __floats2half2_rn(x, y);
              p[i >> 1] = *reinterpret_cast<const uint32_t*>(&h);
            }
            tc_st16(trow + j * 16, p);  // over columns that this thread has read
          }
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          if (drafted) {
            // thread = key: value rows past the end hold anything, a node's value that is not finite must not meet
            // another branch's zero weights: zero them; its descendants get it back at the unit's end
            const int slot = k % kS, key = key0 + st;
            alive = __all_sync(0xffffffffu, mbar_wait(&vfull[slot], (k / kS) & 1, abort_flag, a.m.err));
            if (key >= u.ctx) {
              uint8_t* vrow = dsm + SM::kV + slot * SM::kTile + st * 128;
#pragma unroll 4
              for (int i = 0; i < D / 8; ++i) {
                uint4* p = reinterpret_cast<uint4*>(vrow + (i >> 3) * SM::kPanel + (i & 7) * 16);
                uint4 x = *p;
                uint32_t* w = reinterpret_cast<uint32_t*>(&x);
                bool change = false;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  if (key >= end) {
                    change = true;
                    w[z] = 0u;
                  } else {
                    const uint32_t mk = ((w[z] & 0x7C00u) == 0x7C00u ? 0xFFFFu : 0u) |
                                        ((w[z] & 0x7C000000u) == 0x7C000000u ? 0xFFFF0000u : 0u);
                    if (mk) {
                      w[z] &= ~mk;
                      change = true;
                      flags[1] = 1;
                    }
                  }
                }
                if (change) *p = x;
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          tc_wait_st();
          tc_fence_before();
        }
        mbar_arrive(pfull);
      }
      // ---- the unit's rows: final, or this CTA's record ----
      alive = __all_sync(0xffffffffu, alive && mbar_wait(ofull, n_unit & 1, abort_flag, a.m.err));
      group_bar();
      if (alive) {
        tc_fence_after();
        const bool odd = *reinterpret_cast<volatile int*>(flags + 1) != 0, whole = t0 == 0 && t1 == u.tiles;
        float* rec = tree_record(a, blockIdx.x, t0 == 0);
        const int row = u.row_tile * kTR + r;
        const int j0 = max(t0 * kTK - u.ctx, 0), j1 = min(t1 * kTK - u.ctx, u.nodes);
        const bool zero = l == 0.f || __ldg(a.m.pos + node) < 0;
        const float inv = whole ? 1.0f / l : 1.0f;
        const int64_t off = node * a.ldo + (int64_t)(u.head * G + row % G) * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          uint32_t o[32];
          tc_ld32(trow + 128 + j * 32, o);
          if (r < rows) {
            if (odd) {  // rare: the values that were taken out, for the rows that see them
              const int32_t* table = a.m.tables + __ldg(a.m.tab_start + u.seq);
              for (int n = j0; n < j1; ++n) {
                if (!tree_sees(a.m, node, n)) continue;
                const int p = u.ctx + n;
                const int64_t at = kv_offset(a.layer, __ldg(table + (p >> 4)), 1, u.head, p & 15, a.d.n_blocks, a.d.Hkv, 16, D) + j * 32;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float y = __half2float(reinterpret_cast<const __half*>(a.kv)[at + i]);
                  if (!isfinite(y)) o[i] = __float_as_uint(__uint_as_float(o[i]) + y);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4 v = make_float4(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv,
                                     __uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
              if (whole) tree_store4(a.out, a.out_type, off + j * 32 + i, zero ? make_float4(0.f, 0.f, 0.f, 0.f) : v);
              else *reinterpret_cast<float4*>(rec + r * D + j * 32 + i) = v;
            }
          }
        }
        if (!whole && r < rows) {
          rec[kTR * D + r] = m;
          rec[kTR * D + kTR + r] = l;
        }
        tc_fence_before();  // O has been read before the next unit's first P is announced
      }
      group_bar();
      if (st == 0) flags[1] = 0;
      group_bar();
      left -= t1 - t0;
      tile = 0;
      if (left > 0) tree_unit_next(a.m, G, kTR, a.d.Hkv, u);
    }
  }

  __syncthreads();
  // the last commit has arrived (every MMA and every commit before it has); after an abort also the copies in flight
  const uint64_t w0 = global_ns();
  if (warp == 1)
    while (!mbar_try(mma_done, 0) && global_ns() - w0 < kWaitLimitNs) {
    }
  if (threadIdx.x == 0 && *abort_flag)
    for (int i = max(flags[3] - 2 * kS, 0); i < flags[3]; ++i) {
      uint64_t* f = (i & 1) ? &vfull[(i >> 1) % kS] : &kfull[(i >> 1) % kS];
      while (!mbar_try(f, ((i >> 1) / kS) & 1) && global_ns() - w0 < kWaitLimitNs) {
      }
    }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

template <int D>
cudaError_t one(const TreeAttendArgs& a, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  static SmemOptIn opt;
  constexpr int smem = TcSmem<D>::kBytes;
  static_assert(smem <= 115712, "two CTAs per SM");
  cudaError_t e = opt.ensure(k_tree_attend_tc<D>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_attend_tc<D>, ctas, kTcTreeThreads, smem, s, *tm, a);
}

}  // namespace

cudaError_t launch_tree_attend_tc(const TreeAttendArgs& a, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  switch (a.d.D) {
    case 64: return one<64>(a, tm, ctas, s);
    case 128: return one<128>(a, tm, ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dec
