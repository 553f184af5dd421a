// kernels_tree_tc.cu - tree attention over an f16 or 8-bit cache for wide trees,
// on the 5th-generation tensor cores (tcgen05, accumulators in TMEM).
//
// The same formula as kernels_tree_f16.cu with 128 keys and 128 or 256 rows
// (nodes x query heads of one KV head) per step, one CTA per SM:
//   warps 0..7    two softmax groups of 128 threads, each with its own S and O
//                 in TMEM: thread = row = TMEM lane.  S is read from TMEM, the
//                 weights go back as f16 over the first half of its columns; a
//                 row's maximum and sum never leave their thread
//   warp 8        TMA producer: K and V tiles of 128 keys, 128-byte swizzled
//                 rows of 64 channels, the panels of eight keys side by side
//                 (one box of 4 KB per block: with one per block and panel the
//                 copies' issue alone took 0.75 us for 32 KB: 32 x 64 nodes over
//                 1024-2048 keys took 53.8 us, now 50.9),
//                 into a ring of tile slots, K and V of a tile in turn
//   warp 9        issues S = Q K^T (both operands K-major in shared memory) and
//                 O += P V (P from TMEM, V as a channel-major operand: its
//                 panels are read transposed by the MMA itself), always with a
//                 group's next S queued while the other group's softmax runs
//   warps 10, 11  narrow: the next unit's queries into the other of two buffers;
//                 11: publishes the part of a unit that another CTA joins
// Narrow (up to 128 rows): the groups take the key tiles of the same rows in
// turn and join their halves at the unit's end, each for half of the channels.
// Wide: group b takes rows 128 b .. 128 b + 127 of every tile, so a tile's bytes
// serve 256 rows; with narrow units 8 x 256 nodes at contexts of 8000 read
// every key four times and ran at HBM speed, 211 us against 64 for the products.
// O is rescaled in TMEM only when a row's scores exceed its reference by 2^8, of
// 8 bits 2^15 (exact: numerator and denominator share the reference).  Warps whose rows are
// all behind the last skip the softmax.  Roundings as in kernels_tree_f16.cu.
//
// 8-bit caches: the producer brings codes (a page is contiguous: one bulk copy)
// into a ring of their own, and
//   warps 12..15  turn them into f16 operand tiles of the layout above.
// A tile of 128 keys takes 2^A out of its keys, A near the largest K exponent of
// its eight blocks, and 2^B of V's out of its values: an operand is code * 2^(a -
// A), one fused multiply-add on the way from i8 to f16, exact down to 2^-24.  The
// largest page keeps a factor of 2^5 (i8; e4m3: 2^7, f16's range allows that
// much), so operands are exact while K's scales lie within 2^29 (e4m3, whose codes
// end at 2^-9: 2^22).  So the softmax has one factor c 2^A
// and one exponent B a tile: weights are 2^(s + B - m), l adds 2^-B times their
// sum (the reference m as in kernels_tree_q8.cu).  With a factor for each block
// in the softmax it took 1.3 us a tile in place of 0.85.
// The largest s + B may then pass a row's true one, the largest s + b, by as much
// as the V exponents of a tile differ (a page of large values whose weights are
// all small).  Up to 2^8 the reference makes up for it: it is set 2^8 below that
// largest and raised once weights would pass 2^15 (f16 ends at 2^16), so a row's
// largest true weight is 1 or more, as in kernels_tree_q8.cu, and weights down to
// 2^-14 of it keep all their bits.  A tile whose pages lie further apart (K's or
// V's) takes each block's own 2^a and b into the scores, its K codes as they are,
// and its V codes all times the power of two that other tiles give to their largest
// page, so that B and b mean the same.
// Registers are moved from the other warps to the softmax (512 threads have 128
// each).  32 x 64 nodes over 1024-2048 keys: 52.7 us, 119 MB at 2.3 TB/s; 8 x 256
// over 8000: 137 us, 927 TFLOP/s.  Neither the codes' bytes nor the products bound
// it but the steps of a tile, one after the other, with a conversion more than over
// f16: there the same calls take up to a sixth less time.  The wide form spills: 20
// bytes at head_dim 128, 140 (e4m3: 44) at 64.
#include "attn_fold.cuh"
#include "q8.cuh"
#include "tc_common.cuh"

namespace dec {

namespace {

constexpr int kTR = 128, kTK = 128;  // rows and keys of a step
constexpr int kTcTreeThreads = 384, kTcTreeThreadsQ8 = 512;
// A tile's 2^A, B (infinite: pages far apart), its blocks' b, reckoned as B is, and their 2^a; of how many tiles they are
// kept (the conversion is at most four ahead of the softmax)
struct TileScales {
  float a, b, each[8], keys[8];
};
constexpr int kScaleRing = 8, kApart = 8;
// Of 8 bits: how far below the largest score a reference is set, and how far above it scores may lie
constexpr float kBelow8 = (float)kApart, kAbove8 = 15.f;
constexpr int kOps8 = 3, kSlots8 = 4;  // of 128 channels
constexpr uint32_t kTmemCols = 512;  // S of the two groups: columns 0, 128; O: 256, 256 + D

template <int D, bool kQ8>
struct TcSmem {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = kTR * 128;            // bytes of 64 channels of 128 queries
  static constexpr int kGroup = kPanels * 1024;       // bytes of eight keys
  static constexpr int kTile = kPanels * kPanel;
  // operand tiles (at least K, V, K are in use at once) and, for 8 bits, slots for codes; else the copies land in the operands
  static constexpr int kOps = kQ8 ? (D == 128 ? kOps8 : 2 * kOps8) : D == 128 ? 5 : 10;
  static constexpr int kSlots = kQ8 ? (D == 128 ? kSlots8 : 2 * kSlots8) : kOps;
  static constexpr int kQ = 0;                        // two tiles: the units' in turn (narrow), the groups' (wide)
  static constexpr int kRing = 2 * kTile, kCodes = kRing + kOps * kTile, kCodeTile = kTK * D;
  static constexpr int kFac = kCodes + (kQ8 ? kSlots * kCodeTile : 0);  // float [2][kTR], as the queries
  static constexpr int kScales = kFac + 2 * kTR * 4;                    // TileScales [kScaleRing]
  static constexpr int kBar = kScales + (kQ8 ? kScaleRing * (int)sizeof(TileScales) : 0);
  // barriers: full, empty [slots]; ready, used [operands] of 8 bits; Q full, Q empty, S full, P full, O full, O empty [2]; MMA done
  static constexpr int kBars = 2 * kSlots + (kQ8 ? 2 * kOps : 0) + 15;
  static constexpr int kBytes = kBar + kBars * 8 + 32;
};

__device__ __forceinline__ void tma_box_5d(void* dst, const CUtensorMap* map, int group, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(group), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// One MMA, operands' descriptors as halves: along K only the low one moves (its
// address field, in 16-byte units), so a step is one 32-bit addition each.
// D (TMEM) += A (shared memory) B (shared memory)
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t a_hi, uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}
// D (TMEM) += A (TMEM, f16 pairs per column) B (shared memory)
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}

// Instruction descriptor, kind::f16: f16 operands, fp32 accumulator; bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 128-byte swizzled operand in groups of 8 keys, `group` bytes apart.  Keys along N (K-major): the first 64 channels, more
// of them a panel's 1024 bytes on.  Keys along K (MN-major): panels of 64 channels 1024 bytes apart.
__device__ __forceinline__ uint64_t keys_desc(uint32_t saddr, uint32_t group, bool mn) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(mn ? 1024 >> 4 : 1) << 16) | ((uint64_t)(group >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// A load that runs on: its values are there after the next tc_wait32 on them.
__device__ __forceinline__ void tc_ld32_async(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_wait32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                 "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                 "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
// 16 columns, there when it returns.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// A tile of 128 keys' codes (rows of D bytes) as an operand, by 128 threads: thread t's row and 16-byte chunk of round i.
// Eight lanes of an access take four chunks of a row and the other four (D = 64: the same) of its neighbour, so that reads
// and writes touch every bank once.  The rows of a round lie in one block (D = 64: a warp's).
template <int D>
__device__ __forceinline__ void tc_chunk(int i, int t, int& r, int& c) {
  if constexpr (D == 128) {
    r = i * 16 + (t >> 4) * 2 + ((t >> 2) & 1);
    c = (t & 3) + 4 * (((t >> 2) ^ (t >> 3)) & 1);
  } else {
    r = i * 32 + (t >> 2);
    c = t & 3;
  }
}

template <int D, bool kWide, int kKind>
__global__ void __launch_bounds__(kKind == kTreeF16 ? kTcTreeThreads : kTcTreeThreadsQ8, 1)
    k_tree_attend_tc(const __grid_constant__ CUtensorMap tm, const __grid_constant__ TreeAttendArgs a) {
  constexpr bool kQ8 = kKind != kTreeF16;
  using SM = TcSmem<D, kQ8>;
  constexpr int kS = SM::kSlots, kOps = SM::kOps, kR = kWide ? 2 * kTR : kTR;
  // of 8 bits: 256 threads each, in all the 512 x 128 of the launch.  Narrow (152 / 104, 160 / 96): 32 x 64 nodes over
  // 1024-2048 keys 53.5, 52.4 us, 1 x 64 over 40000 41.5, 40.9; wide: 8 x 256 over 8000 135.9, 140.3
  constexpr int kSoftmaxRegs = kWide ? 152 : 160, kOtherRegs = 256 - kSoftmaxRegs;
  extern __shared__ __align__(1024) uint8_t dsm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsm + SM::kBar);
  // ready, used: of the operands that the MMAs take (an f16 cache's copies are these)
  uint64_t *full = bars, *empty = bars + kS, *ready = kQ8 ? bars + 2 * kS : full, *used = kQ8 ? ready + kOps : empty,
           *qfull = kQ8 ? used + kOps : bars + 2 * kS, *qempty = qfull + 2, *sfull = qfull + 4,
           *pfull = qfull + 6, *ofull = qfull + 8, *oempty = qfull + 10, *mma_done = qfull + 12, *phalf = qfull + 13;
  // [0] abort, [1] TMEM base, [2] slots filled, [4 + i] 1 + the unit (of parity i) that met a value that is not finite
  int* flags = reinterpret_cast<int*>(bars + SM::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kQ8 ? 4 : 1);
    }
    for (int i = 0; kQ8 && i < kOps; ++i) {
      mbar_init(&ready[i], 4);
      mbar_init(&used[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], kWide ? 128 : 320);
      mbar_init(&qempty[i], 256);
      mbar_init(&sfull[i], kQ8 ? 2 : 1);
      mbar_init(&pfull[i], 128);
      mbar_init(&phalf[i], 128);
      mbar_init(&ofull[i], 1);
      mbar_init(&oempty[i], kWide ? 128 : 256);
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < 8; ++i) flags[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the plan is older than the kernels before this one: read before they are waited for
  const int here = tree_place();
  const TreeCut cut = a.m.cuts[here];
  const bool ok_shape = tree_shape_ok(a.m, true);
  TreeUnit u = tree_unit_first(a.m, cut);
  int tile = cut.tile, n_unit = 0;
  // a lane's block of tile t, if that is in front of t1
  auto entry = [&](int t, int t1) {
    const int b = t * 8 + (lane & 7);
    int blk = b < (u.ctx + u.nodes + 15) >> 4 && t < t1 ? __ldg(a.m.tables + u.tab + b) : 0;
#ifdef DEC_DEBUG
    if ((unsigned)blk >= (unsigned)a.d.n_blocks) {
      atomicOr(a.m.err, kErrBounds);
      blk = 0;
    }
#endif
    return blk;
  };
  // a lane's block of the four tiles from t on
  auto entry4 = [&](int t, int t1) { return entry(t + (lane >> 3), t1); };
  int nxt = 0;
  if (ok_shape && cut.count > 0) {
    const int t1 = min(u.tiles, tile + cut.count);
    if (warp == 8) nxt = entry(tile, t1);
    else if (kQ8 && warp >= 12) nxt = entry4(tile, t1);
  }
  __syncthreads();
  // the tensor memory, too, before the wait
  if (warp == 9 && ok_shape) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(flags + 1)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait_prev();
  pdl_launch_next();
  if (!ok_shape) return;
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(flags + 1);
  volatile int* abort_flag = flags;
  // (the softmax warps raise theirs in their own branch: where branches meet the compiler counts on the fewest)
  if (kQ8 && warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  const int gs = a.d.gs, G = 1 << gs;
  // a wide unit with at most 128 rows leaves the second group out
  auto both = [&](const TreeUnit& x) { return (x.nodes << gs) - x.row_tile * kR > kTR; };

  if (warp == 8) {
    // ---- producer: lanes 0..7 copy a block each, K, then V ----
    int li = 0;  // loads so far: K of tile k is load 2k, V is 2k + 1
    for (int left = cut.count; left > 0;) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), blocks = (u.ctx + u.nodes + 15) >> 4;
      if (left < cut.count) nxt = entry(t0, t1);  // the first unit's is there
      for (int t = t0; t < t1; ++t) {
        const int here = min(8, blocks - t * 8), blk = nxt;
        nxt = entry(t + 1, t1);
        const uint32_t bytes = here * (kQ8 ? 16 * D : SM::kPanels * 2048);
        const int z = (a.layer * a.d.n_blocks + blk) * 2;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v, ++li) {
          const int slot = li % kS;
          bool ok = true;
          if (lane == 0 && li >= kS) ok = mbar_wait(&empty[slot], ((li / kS) - 1) & 1, abort_flag, a.m.err);
          if (!__shfl_sync(0xffffffffu, (int)ok, 0)) goto produced;
          if (lane == 0) {
            mbar_expect_tx(&full[slot], bytes);
            flags[2] = li + 1;
          }
          __syncwarp();
          if constexpr (kQ8) {
            if (lane < here)
              bulk_g2s(dsm + SM::kCodes + slot * SM::kCodeTile + lane * 16 * D,
                       reinterpret_cast<const uint8_t*>(a.kv) + kv_offset(a.layer, blk, is_v, u.head, 0, a.d.n_blocks, a.d.Hkv, 16, D), 16 * D, &full[slot]);
          } else if (lane < here)
            tma_box_5d(dsm + SM::kRing + slot * SM::kTile + lane * 2 * SM::kGroup, &tm, u.head * 2, z + is_v, &full[slot]);
          __syncwarp();
        }
      }
      left -= t1 - t0;
      tile = 0;
      if (left > 0) tree_unit_next(a.m, gs, kR, a.d.Hkv, u);
    }
  produced:;
  } else if (warp == 9) {
    // ---- MMA issuer: the whole warp walks the tiles, one elected lane issues.  Everything that the MMAs' operands and the
    // loops go by is broadcast, so that the compiler keeps it in uniform registers, where the MMAs take their operands from ----
    constexpr uint32_t id_s = idesc_f16(kTR, kTK, false), id_o = idesc_f16(kTR, D, true);
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    auto wait = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, abort_flag, a.m.err)) != 0;
    };
    uint32_t leader;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
    const uint32_t td = uni(tmem), smem0 = uni(smem_u32(dsm));
    const uint64_t q_desc = sw128_desc(smem0 + SM::kQ);
    const uint64_t k_desc = keys_desc(smem0 + SM::kRing, SM::kGroup, false), v_desc = keys_desc(smem0 + SM::kRing, SM::kGroup, true);
    const uint32_t q_hi = (uint32_t)(q_desc >> 32), q_lo = (uint32_t)q_desc;
    const uint32_t hi = (uint32_t)(k_desc >> 32), k_lo = (uint32_t)k_desc, v_lo = (uint32_t)v_desc;  // V's high half is K's
    // the copies of load li (K of tile k: 2 k, V: 2 k + 1) have landed
    auto landed = [&](int li) { return wait(&ready[li % kOps], li / kOps); };
    // scores of tile k (landed) into group b's S, from query tile q
    auto scores = [&](int k, int b, int q, bool last) {
      const int slot = 2 * k % kOps;
      const uint32_t qd = q_lo + q * (SM::kTile >> 4), kd = k_lo + slot * (SM::kTile >> 4);
      if (leader) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t in = (i & 3) * 32;
          mma_ss(td + b * 128, qd + (((i >> 2) * SM::kPanel + in) >> 4), kd + (((i >> 2) * 1024 + in) >> 4), q_hi, hi, id_s, i != 0);
        }
        tc_commit(&sfull[b]);
        if (last) tc_commit(&used[slot]);
        if constexpr (kQ8) mbar_arrive(&sfull[b]);  // the tile's scales, which this warp has acquired with the operand
      }
    };
    // weights (tile n of group b) times values of tile k (landed)
    auto values = [&](int k, int b, int n, bool fresh, bool last) -> bool {
      const int slot = (2 * k + 1) % kOps;
      const uint32_t vd = v_lo + slot * (SM::kTile >> 4);
      constexpr int kHalf = kWide ? 0 : kTK / 32;
      // narrow: the first half of the keys while the second's weights are worked on (32 x 64: 50.9 us, so 50.5; 8 x 256 took
      // 134 us with it instead of 114: the issuer then waits for one group while the other one is ready)
      if constexpr (!kWide) {
        if (!wait(&phalf[b], n)) return false;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i)
            mma_ts(td + 256 + b * D, td + b * 128 + i * 8, vd + i * (2 * SM::kGroup >> 4), hi, id_o, i != 0 || !fresh);
        }
        __syncwarp();
      }
      if (!wait(&pfull[b], n)) return false;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int i = kHalf; i < kTK / 16; ++i)
          mma_ts(td + 256 + b * D, td + b * 128 + i * 8, vd + i * (2 * SM::kGroup >> 4), hi, id_o, i != 0 || !fresh);
        if (last) tc_commit(&used[slot]);
      }
      return true;
    };
    const int count = uni(cut.count);
    int k = 0;
    if constexpr (!kWide) {
      auto tile_scores = [&](int x, int unit, bool first) -> bool {
        if (!landed(2 * x) || (first && !wait(&qfull[unit & 1], unit >> 1))) return false;
        tc_fence_after();
        scores(x, x & 1, unit & 1, true);
        return true;
      };
      bool ok = count == 0 || tile_scores(0, 0, true);
      for (int left = count; ok && left > 0; ++n_unit) {
        const int tiles = uni(min(u.tiles - tile, left));
        int fresh = 3;  // groups whose O this unit has not written yet
        for (int t = 0; ok && t < tiles; ++t, ++k) {
          const int b = k & 1;
          // the unit's next scores first; O once the unit before has been read out of it.  (The next unit's first scores
          // wait for keys that may be far off: ahead of this unit's last values they held up its end, 54.4 us against 53.8)
          ok = (t + 1 == tiles || tile_scores(k + 1, n_unit, false)) && landed(2 * k + 1) &&
               (t > 0 || n_unit == 0 || wait(&oempty[0], n_unit - 1)) && values(k, b, k >> 1, (fresh >> b) & 1, true);
          fresh &= ~(1 << b);
        }
        if (!ok) break;
        if (leader) tc_commit(&ofull[0]);
        left -= tiles;
        tile = 0;
        if (left > 0) {
          tree_unit_next(a.m, gs, kR, a.d.Hkv, u);
          ok = tile_scores(k, n_unit + 1, true);
        }
      }
    } else {
      int n0 = 0, n1 = 0, units0 = 0, units1 = 0;  // tiles and units of each group
      int groups = uni(both(u) ? 2 : 1);
      bool ok = true;
      // the scores of a unit's first tile
      auto first_scores = [&](int x) -> bool {
        if (!landed(2 * x) || !wait(&qfull[0], units0)) return false;
        tc_fence_after();
        scores(x, 0, 0, groups == 1);
        if (groups == 1) return true;
        if (!wait(&qfull[1], units1)) return false;
        tc_fence_after();
        scores(x, 1, 1, true);
        return true;
      };
      if (count > 0) ok = first_scores(0);
      for (int left = count; ok && left > 0;) {
        const int tiles = uni(min(u.tiles - tile, left));
        if (units0 > 0) ok = wait(&oempty[0], units0 - 1);
        if (groups == 2 && units1 > 0) ok = ok && wait(&oempty[1], units1 - 1);
        for (int t = 0; ok && t < tiles; ++t, ++k) {
          const bool more = t + 1 < tiles;
          // both copies are waited for ahead of the weights: from there to a group's next scores nothing else is in the way
          ok = landed(2 * k + 1) && (!more || landed(2 * k + 2)) && values(k, 0, n0++, t == 0, groups == 1);
          if (!ok) break;
          if (more) scores(k + 1, 0, 0, groups == 1);
          else if (leader) tc_commit(&ofull[0]);
          if (groups == 1) continue;
          ok = values(k, 1, n1++, t == 0, true);
          if (!ok) break;
          if (more) scores(k + 1, 1, 1, true);
          else if (leader) tc_commit(&ofull[1]);
        }
        if (!ok) break;
        ++units0;
        units1 += groups - 1;
        left -= tiles;
        tile = 0;
        if (left > 0) {
          tree_unit_next(a.m, gs, kR, a.d.Hkv, u);
          groups = uni(both(u) ? 2 : 1);
          ok = first_scores(k);
        }
      }
    }
    if (leader) tc_commit(mma_done);
    __syncwarp();
  } else if (kQ8 && warp >= 12) {
    // ---- codes to operands ----
    constexpr int kLift = kKind == kTreeI8 ? 5 : 7;  // 1152 2^5 and 448 2^7 are still f16
    // how far K's exponents may lie apart: codes are multiples of 1 (e4m3: 2^-9), f16 numbers of 2^-24
    constexpr int kApartKeys = kLift + 24 - (kKind == kTreeI8 ? 0 : 9);
    const int ct = threadIdx.x - 384;
    int li = 0;
    for (int left = cut.count; left > 0;) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), blocks = (u.ctx + u.nodes + 15) >> 4;
      if (left < cut.count) nxt = entry4(t0, t1);  // the first unit's are there
      // exponents of K and V of a lane's block of four tiles, if it is one; the next tiles' are loaded before the last of these
      // is worked on
      int2 e;
      bool block = false;
      auto exponents = [&](int t, int blk) {
        const int x = t + (lane >> 3);
        e = make_int2(kExpMin, kExpMin);
        block = x < t1 && x * 8 + (lane & 7) < blocks;
        if (block) {
          const float2 y = *reinterpret_cast<const float2*>(a.scales + q8_scale_at(a.d, a.layer, blk, u.head, 0));
          e = make_int2(q8_exp(y.x), q8_exp(y.y));
        }
      };
      exponents(t0, nxt);
      uint32_t fk = 0, fv = 0;  // the factors of the lane's block, in both halves
      TileScales scales;        // of its tile (each[0]: the block's)
      for (int t = t0; t < t1; ++t) {
        const int turn = (t - t0) & 3;
        if (turn == 0) {
          nxt = entry4(t + 4, t1);
          int ka = e.x, va = e.y, klow = block ? e.x : kExpMax, low = block ? e.y : kExpMax;
#pragma unroll
          for (int d = 1; d < 8; d *= 2) {
            ka = max(ka, __shfl_xor_sync(0xffffffffu, ka, d));
            va = max(va, __shfl_xor_sync(0xffffffffu, va, d));
            klow = min(klow, __shfl_xor_sync(0xffffffffu, klow, d));
            low = min(low, __shfl_xor_sync(0xffffffffu, low, d));
          }
          const bool apart = va - low > kApart || ka - klow > kApartKeys;
          scales.a = q8_two(ka - kLift);
          scales.b = apart ? INFINITY : (float)(va - kLift);
          scales.each[0] = (float)(e.y - kLift);
          scales.keys[0] = q8_two(e.x);
          // 2^d in f16, down to 2^-24 (below, 0)
          auto half_two = [](int d) { return (d >= -14 ? (uint32_t)(d + 15) << 10 : d >= -24 ? 1u << (d + 24) : 0u) * 0x10001u; };
          fk = half_two(apart ? 0 : e.x - ka + kLift);
          fv = half_two(apart ? kLift : e.y - va + kLift);
        }
        if (warp == 12 && lane >> 3 == turn) {
          TileScales& to = reinterpret_cast<TileScales*>(dsm + SM::kScales)[(li >> 1) % kScaleRing];
          to.each[lane & 7] = scales.each[0];
          to.keys[lane & 7] = scales.keys[0];
          if ((lane & 7) == 0) to.a = scales.a, to.b = scales.b;
        }
        if (turn == 3) exponents(t + 1, nxt);
        const bool odd = t * kTK + kTK > u.ctx;  // rows of no token among them, perhaps
#pragma unroll 1
        for (int is_v = 0; is_v < 2; ++is_v, ++li) {
          const int slot = li % kS, op = li % kOps;
          bool ok = mbar_wait(&full[slot], (li / kS) & 1, abort_flag, a.m.err);
          if (!__all_sync(0xffffffffu, ok)) goto converted;
          ok = li < kOps || mbar_wait(&used[op], ((li / kOps) - 1) & 1, abort_flag, a.m.err);
          if (!__all_sync(0xffffffffu, ok)) goto converted;
          const uint32_t f = is_v ? fv : fk;
          int r, c;
          tc_chunk<D>(0, ct, r, c);
          // a round's rows lie 16 (D = 64: 32) below the last one's: the same place in their group, two (four) groups on
          const uint8_t* from = dsm + SM::kCodes + slot * SM::kCodeTile + r * D + c * 16;
          uint8_t* to8 = dsm + SM::kRing + op * SM::kTile + (r >> 3) * SM::kGroup + (c >> 2) * 1024 + (r & 7) * 128;
          const int x0 = ((c & 3) * 2 ^ (r & 7)) << 4, x1 = (((c & 3) * 2 + 1) ^ (r & 7)) << 4;
          constexpr int kRows = D == 128 ? 16 : 32, kU = 4;
#pragma unroll 1
          for (int i = 0; i < D / 16; i += kU) {
            uint4 raw[kU];
#pragma unroll
            for (int y = 0; y < kU; ++y) raw[y] = *reinterpret_cast<const uint4*>(from + (i + y) * kRows * D);
#pragma unroll
            for (int y = 0; y < kU; ++y) {
              const uint32_t two = __shfl_sync(0xffffffffu, f, turn * 8 + (D == 128 ? i + y : (i + y) * 2 + (ct >> 6)));
              uint32_t w[4] = {raw[y].x, raw[y].y, raw[y].z, raw[y].w}, h[8];
              if (kKind == kTreeE4m3 && odd) {
#pragma unroll
                for (int z = 0; z < 4; ++z) w[z] = e4m3_numbers(w[z]);
              }
#pragma unroll
              for (int z = 0; z < 4; ++z) q8_halves_times<kKind>(w[z], two, h[2 * z], h[2 * z + 1]);
              uint8_t* at = to8 + (i + y) * (kRows / 8) * SM::kGroup;
              *reinterpret_cast<uint4*>(at + x0) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(at + x1) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&empty[slot]);
            mbar_arrive(&ready[op]);
          }
        }
      }
      left -= t1 - t0;
      tile = 0;
      if (left > 0) tree_unit_next(a.m, gs, kR, a.d.Hkv, u);
    }
  converted:;
  } else if (warp >= 10) {
    // ---- Queries one unit ahead (the first unit's by the softmax warps, which have nothing else to do yet).
    // One of these warps also publishes the part of a shared unit that this CTA begins with: the fence takes up to 3 us
    // under load, and the softmax warps have the next unit to go on with.  ----
    bool publish = warp == 11 && cut.awaited;
    auto published = [&]() {
      asm volatile("bar.sync 4, 288;" ::: "memory");
      if (lane == 0) tree_publish(a.m, here);
      publish = false;
    };
    for (int left = kWide ? 0 : cut.count; left > 0; ++n_unit) {
      const int b = n_unit & 1;
      if (publish && n_unit == 2) published();  // the first two units' queries are on their way
      if (!__all_sync(0xffffffffu, n_unit < 2 || mbar_wait(&qempty[b], ((n_unit >> 1) - 1) & 1, abort_flag, a.m.err))) break;
      if (n_unit > 0)
        tree_load_queries<D, kTR, 2, 4>(a, u, u.row_tile * kTR, warp - 10, reinterpret_cast<float*>(dsm + SM::kFac) + b * kTR, [&](int q, int x, uint4 h) {
          *reinterpret_cast<uint4*>(dsm + SM::kQ + b * SM::kTile + (x >> 3) * SM::kPanel + q * 128 + (((x & 7) ^ (q & 7)) << 4)) = h;
        });
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&qfull[b]);
      left -= min(u.tiles, tile + left) - tile;
      tile = 0;
      if (left > 0) tree_unit_next(a.m, gs, kR, a.d.Hkv, u);
    }
    if (publish) published();
  } else {
    if constexpr (kQ8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax ----
    const int b = warp >> 2, wr = (warp & 3) * 32, r = wr + lane, st = threadIdx.x & 127;
    const int row_in = (kWide ? b * kTR : 0) + r;  // row of the unit
    const uint32_t trow = tmem + ((uint32_t)wr << 16), ts = trow + b * 128, to = trow + 256 + b * D;
    float* fac = reinterpret_cast<float*>(dsm + SM::kFac);
    auto group_bar = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(2 + b) : "memory"); };
    // wide: this group's queries of unit x
    auto load_group = [&](const TreeUnit& x) {
      tree_load_queries<D, kTR, 4, 8>(a, x, x.row_tile * kR + b * kTR, warp & 3, fac + b * kTR, [&](int q, int c, uint4 h) {
        *reinterpret_cast<uint4*>(dsm + SM::kQ + b * SM::kTile + (c >> 3) * SM::kPanel + q * 128 + (((c & 7) ^ (q & 7)) << 4)) = h;
      });
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&qfull[b]);
    };
    int k = 0, n = 0, units = 0;  // tiles; of this group: tiles and units
    const bool out16 = ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(a.ldo * 2)) & 15) == 0;  // rows in 16-byte pieces
    bool alive = true;
    if (cut.count > 0) {
      if constexpr (kWide) {
        if (b == 0 || both(u)) load_group(u);
      } else {
        tree_load_queries<D, kTR, 8, 8>(a, u, u.row_tile * kTR, warp, fac, [&](int q, int x, uint4 h) {
          *reinterpret_cast<uint4*>(dsm + SM::kQ + (x >> 3) * SM::kPanel + q * 128 + (((x & 7) ^ (q & 7)) << 4)) = h;
        });
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(&qfull[0]);
      }
    }
    for (int left = cut.count; left > 0; ++n_unit) {
      const int t0 = tile, t1 = min(u.tiles, tile + left), end = u.ctx + u.nodes, k0 = k;
      const int row = u.row_tile * kR + row_in, all_rows = u.nodes << gs;
      const bool mine = row - lane < all_rows;  // some row of this warp is one
      const bool in = !kWide || b == 0 || both(u);
      const int node = u.node0 + min(row >> gs, u.nodes - 1);
      const uint32_t* anc = a.m.anc + (size_t)node * a.m.words;
      const bool pad = __ldg(a.m.pos + node) < 0;
      float c = 0.f, m = -INFINITY, l = 0.f;
      if (in) {
        if constexpr (kWide) {
          group_bar();  // the factors of the group's queries
          c = fac[b * kTR + r];
        } else {
          alive = __all_sync(0xffffffffu, alive && mbar_wait(&qfull[n_unit & 1], (n_unit >> 1) & 1, abort_flag, a.m.err));
          c = fac[(n_unit & 1) * kTR + r];
          mbar_arrive(&qfull[(n_unit + 1) & 1]);  // the next unit's queries come from the other warps alone
        }
      }
      bool first = true;
      for (int t = t0; t < t1; ++t, ++k) {
        if (!in || (!kWide && (k & 1) != b)) continue;
        const int key0 = t * kTK;
        const bool drafted = key0 + kTK > u.ctx;
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};  // keys of each 32 that this row sees
        if (drafted) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int x = key0 + j * 32 - u.ctx;  // node number of the first; negative: cached tokens
            const int w = x >> 5;
            const uint32_t lo = x > -32 && w < a.m.words ? (w < 0 ? 0xffffffffu : __ldg(anc + w)) : 0u;
            const uint32_t hi = x > -32 && w + 1 < a.m.words ? __ldg(anc + w + 1) : 0u;
            if (x > -32) vis[j] = __funnelshift_r(lo, hi, x & 31);
          }
          // value rows past the end hold anything, a node's value that is not finite must not meet another branch's
          // zero weights: zero them; its descendants get it back at the unit's end.  Eight threads per row.  (Wide: both
          // groups do this for the tile, whichever comes first changes it.  8 bits: operands are always finite)
          if constexpr (!kQ8) {
            const int li = 2 * k + 1, slot = li % kS;
            alive = __all_sync(0xffffffffu, alive && mbar_wait(&full[slot], (li / kS) & 1, abort_flag, a.m.err));
            for (int q = max(u.ctx - key0, 0) + (st >> 3); alive && q < kTK; q += 16) {
#pragma unroll
              for (int p = 0; p < SM::kPanels; ++p) {
                uint4* at = reinterpret_cast<uint4*>(dsm + SM::kRing + slot * SM::kTile + (q >> 3) * SM::kGroup + p * 1024 +
                                                     (q & 7) * 128 + (st & 7) * 16);
                uint4 x = *at;
                uint32_t* w = reinterpret_cast<uint32_t*>(&x);
                if (key0 + q >= end) {
                  if (w[0] | w[1] | w[2] | w[3]) *at = make_uint4(0u, 0u, 0u, 0u);
                } else if (tree_not_finite(x)) {
#pragma unroll
                  for (int z = 0; z < 4; ++z) w[z] = tree_finite_or_0(w[z]);
                  *at = x;
                  flags[4 + (n_unit & 1)] = n_unit + 1;
                }
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        alive = __all_sync(0xffffffffu, alive && mbar_wait(&sfull[b], n & 1, abort_flag, a.m.err));
        ++n;
        if (alive && mine) {
          tc_fence_after();
          float f = c, e = 0.f;  // this tile's score factor (8 bits: kept off 0 and infinity, hidden scores are -inf) and exponent
          auto kept = [](float x) { return fminf(fmaxf(x, 1.17549435e-38f), 3.40282347e38f); };
          const TileScales* scales = reinterpret_cast<const TileScales*>(dsm + SM::kScales) + k % kScaleRing;
          bool apart = false;
          if constexpr (kQ8) {
            f = kept(c * scales->a);
            e = scales->b;
            apart = e == INFINITY;
          }
          if (drafted) {  // rare: hide in place what the rows do not see
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
              const uint32_t see = j == 0 ? vis[0] : j == 1 ? vis[1] : j == 2 ? vis[2] : vis[3];
              if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
              uint32_t s[32];
              tc_ld32(ts + j * 32, s);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see >> i) & 1u)) s[i] = 0xff800000u;  // -inf
              tc_st16(ts + j * 32, s);
              tc_st16(ts + j * 32 + 16, s + 16);
            }
            tc_wait_st();
          }
          if (kQ8 && apart) {  // rare: s f + b of each block in place of the scores
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
              const float fb = kept(c * scales->keys[j]), eb = scales->each[j];
              uint32_t s[16];
              tc_ld16(ts + j * 16, s);
#pragma unroll
              for (int i = 0; i < 16; ++i) s[i] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(s[i]), fb), eb));
              tc_st16(ts + j * 16, s);
            }
            tc_wait_st();
            f = 1.f;
            e = 0.f;
          }
          // two passes over S, 32 columns at a time, the next ones on their way while these are worked on (the loops stay
          // loops: unrolled, the tile's code ran out of the instruction cache at every turn)
          uint32_t sa[32], sb[32];
          float mx = -INFINITY;
          auto largest = [&](const uint32_t (&x)[32]) {
            float y[2] = {mx, mx};
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              y[0] = fmaxf(fmaxf(y[0], __uint_as_float(x[i])), __uint_as_float(x[i + 1]));
              y[1] = fmaxf(fmaxf(y[1], __uint_as_float(x[i + 2])), __uint_as_float(x[i + 3]));
            }
            mx = fmaxf(y[0], y[1]);
          };
          tc_ld32_async(ts, sa);
#pragma unroll 1
          for (int j = 0; j < 4; j += 2) {
            tc_wait32(sa);
            tc_ld32_async(ts + j * 32 + 32, sb);
            largest(sa);
            tc_wait32(sb);
            tc_ld32_async(ts + ((j * 32 + 64) & 127), sa);  // at the end the first columns again, for the weights
            largest(sb);
          }
          mx = kQ8 ? __fadd_rn(__fmul_rn(mx, f), e) : mx * f;
          if (__any_sync(0xffffffffu, mx - m > (kQ8 ? kAbove8 : 8.f))) {  // (a sum with m could round up to the next score)
            const float below = mx - (kQ8 ? kBelow8 : 0.f);  // from 2^27 on it may round to 16 below, where weights would be infinite
            const float mn = fmaxf(m, mx - below > kAbove8 ? mx : below), g = mn == m ? 1.f : ex2(m - mn);
            m = mn;
            l *= g;
            if (!first) {  // this group's products so far have run: its S was issued behind them
              tc_wait32(sa);
#pragma unroll 1
              for (int j = 0; j < D / 32; ++j) {
                uint32_t o[32];
                tc_ld32(to + j * 32, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * g);
                tc_st16(to + j * 32, o);
                tc_st16(to + j * 32 + 16, o + 16);
              }
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;
          uint64_t c2 = pack2(f, f), m2 = pack2(e - mu, e - mu), l2[2] = {0ull, 0ull};
          if (kQ8 && apart) {  // the sum, block by block
            tc_wait32(sa);
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
              const float eb = scales->each[j];
              uint32_t s[16];
              tc_ld16(ts + j * 16, s);
              float sum = 0.f;
#pragma unroll
              for (int i = 0; i < 16; ++i) sum += ex2(__uint_as_float(s[i]) - mu);
              l = fmaf(sum, q8_two(-(int)eb), l);
            }
            tc_ld32_async(ts, sa);
          }
          // s c - m in one rounding while the maximum's own (2^-13 up to 2^12) is small against the weights' (2^-11); far out
          // the product is rounded as the maximum was, or the largest score would miss it by its own last place
          if (__any_sync(0xffffffffu, !(fabsf(mu) <= 4096.f))) {
            tc_wait32(sa);
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
              uint32_t s[32];
              tc_ld32(ts + j * 32, s);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = __fmul_rn(__uint_as_float(s[i]), f);
                s[i] = __float_as_uint(__fadd_rn(kQ8 ? __fadd_rn(y, e) : y, -mu));
              }
              tc_st16(ts + j * 32, s);
              tc_st16(ts + j * 32 + 16, s + 16);
            }
            tc_wait_st();
            tc_ld32_async(ts, sa);
            c2 = pack2(1.f, 1.f);
            m2 = 0ull;
          }
          auto weights = [&](const uint32_t (&x)[32], int j) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 z = unpack2(fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, m2));
              const float ex = ex2(z.x), ey = ex2(z.y);
              l2[i & 1] = add2(l2[i & 1], pack2(ex, ey));
              const __half2 hh = __floats2half2_rn(ex, ey);
              p[i] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            tc_st16(ts + j * 16, p);  // over scores that this thread has read
          };
#pragma unroll 1
          for (int j = 0; j < 4; j += 2) {
            tc_wait32(sa);
            tc_ld32_async(ts + j * 32 + 32, sb);
            weights(sa, j);
            tc_wait32(sb);
            if (j == 0) tc_ld32_async(ts + 64, sa);
            weights(sb, j + 1);
            if (!kWide && j == 0) {
              tc_wait_st();
              tc_fence_before();
              mbar_arrive(&phalf[b]);
            }
          }
          const float2 lx = unpack2(add2(l2[0], l2[1]));
          // the weights carry the values' 2^e: take it out (2^-e, whose exponent field is 127 - e)
          if constexpr (!kQ8) l += lx.x + lx.y;
          else if (!apart) l = fmaf(lx.x + lx.y, __uint_as_float(__float_as_uint(8388735.f - e) << 23), l);
          tc_wait_st();
          tc_fence_before();
        } else if constexpr (!kWide) {
          mbar_arrive(&phalf[b]);
        }
        first = false;
        mbar_arrive(&pfull[b]);
      }
      TreeUnit nu = u;
      if (left > t1 - t0) tree_unit_next(a.m, gs, kR, a.d.Hkv, nu);
      if constexpr (kWide) {
        // this group's S of the unit's last tile is there, so its queries are done with: the next unit's, if it takes part
        if (in) group_bar();  // every factor has been read
        if (left > t1 - t0 && (b == 0 || both(nu))) load_group(nu);
      }
      // ---- the unit's end ----
      float L = l, M = m, g0 = 1.f, g1 = 0.f;
      bool has0 = true, has1 = false;
      if (in) alive = __all_sync(0xffffffffu, alive && mbar_wait(&ofull[kWide ? b : 0], units & 1, abort_flag, a.m.err));
      if constexpr (!kWide) {
        // join the two groups, this one for channels b D/2 .. (b + 1) D/2 - 1
        float2* ml = reinterpret_cast<float2*>(dsm + SM::kQ + (n_unit & 1) * SM::kTile);  // the queries are done with
        ml[b * kTR + r] = make_float2(m, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 s0 = ml[r], s1 = ml[kTR + r];
        has0 = t1 - t0 > 1 || (k0 & 1) == 0;
        has1 = t1 - t0 > 1 || (k0 & 1) == 1;
        M = fmaxf(s0.x, s1.x);
        const float mu = M == -INFINITY ? 0.f : M;
        g0 = has0 ? ex2(s0.x - mu) : 0.f;
        g1 = has1 ? ex2(s1.x - mu) : 0.f;
        L = s0.y * g0 + s1.y * g1;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        mbar_arrive(&qempty[n_unit & 1]);
      }
      const bool whole = t0 == 0 && t1 == u.tiles;
      const int follow = !whole && t0 == 0 ? cut.follow : 0;  // CTAs whose parts are joined here
      const bool final = whole || follow;
      if (in && follow) {
        if (st < follow) tree_await(a.m, here + (st + 1) * cut.step);
        group_bar();
      }
      if (in && alive && mine) {
        tc_fence_after();
        const bool odd = !kQ8 && reinterpret_cast<volatile int*>(flags)[4 + (n_unit & 1)] == n_unit + 1;
        const bool valid = row < all_rows;
        float* rec = tree_record(a, here, t0 == 0);
        const int j0 = max(t0 * kTK - u.ctx, 0), j1 = min(t1 * kTK - u.ctx, u.nodes);
        // the parts that are joined: record y - 1's rows, their common maximum and sum
        auto part = [&](int y) -> const float* { return tree_record(a, here + y * cut.step, false); };
        float top = M;
        for (int y = 1; y <= follow; ++y) top = fmaxf(top, __ldcg(part(y) + kR * D + row_in));
        const float mu = top == -INFINITY ? 0.f : top;
        if (follow) {
          const float own = ex2(M - mu);
          L *= own;
          g0 *= own;
          g1 *= own;
          for (int y = 1; y <= follow; ++y) {
            const float* p = part(y) + kR * D + row_in;
            L = fmaf(__ldcg(p + kR), ex2(__ldcg(p) - mu), L);
          }
        }
        const bool zero = L == 0.f || pad;
        const float inv = final ? 1.0f / L : 1.f;
        g0 *= inv;
        g1 *= inv;
        const int64_t off = node * a.ldo + (int64_t)((u.head << gs) + (row & (G - 1))) * D;
        const int ch0 = kWide ? 0 : b * (D / 2), ch1 = kWide ? D : (b + 1) * (D / 2);
        const uint32_t o0 = kWide ? to : trow + 256, o1 = trow + 256 + D;
#pragma unroll 1
        for (int ch = ch0; ch < ch1; ch += 32) {
          uint32_t x[32];
          float v[32];
          if (kWide || has0) {
            tc_ld32(o0 + ch, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(x[i]) * g0;
          }
          if (!kWide && has1) {
            tc_ld32(o1 + ch, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(x[i]), g1, has0 ? v[i] : 0.f);
          }
#pragma unroll 1
          for (int y = 1; y <= follow; ++y) {
            const float f = ex2(__ldcg(part(y) + kR * D + row_in) - mu) * inv;
            const float4* p = reinterpret_cast<const float4*>(part(y)) + (ch / 4) * kR + row_in;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 z = __ldcg(p + i * kR);
              v[4 * i] = fmaf(z.x, f, v[4 * i]);
              v[4 * i + 1] = fmaf(z.y, f, v[4 * i + 1]);
              v[4 * i + 2] = fmaf(z.z, f, v[4 * i + 2]);
              v[4 * i + 3] = fmaf(z.w, f, v[4 * i + 3]);
            }
          }
          if (valid && !final) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)  // whole lines per warp
              reinterpret_cast<float4*>(rec)[((ch + i) / 4) * kR + row_in] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          } else if (valid) {
            uint32_t h[16];
            if (a.out_type == kTreeBf16) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const __nv_bfloat162 z = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                h[i] = *reinterpret_cast<const uint32_t*>(&z);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const __half2 z = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                h[i] = *reinterpret_cast<const uint32_t*>(&z);
              }
            }
            uint16_t* to_out = reinterpret_cast<uint16_t*>(a.out) + off + ch;
            if (zero) {
#pragma unroll
              for (int i = 0; i < 16; ++i) h[i] = 0u;
            }
            if (out16) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) reinterpret_cast<uint4*>(to_out)[i / 4] = make_uint4(h[i], h[i + 1], h[i + 2], h[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 2) reinterpret_cast<uint2*>(to_out)[i / 2] = make_uint2(h[i], h[i + 1]);
            }
          }
          __syncwarp();
        }
        if (odd && valid) {  // rare: the values that were taken out, for the rows that see them
          const int32_t* table = a.m.tables + u.tab;
#pragma unroll 1
          for (int x = j0; x < j1; ++x) {
            if (!tree_sees(a.m, node, x)) continue;
            const int p = u.ctx + x;
            const __half* at = reinterpret_cast<const __half*>(a.kv) +
                               kv_offset(a.layer, tree_block(a.m, a.d.n_blocks, __ldg(table + (p >> 4))), 1, u.head, p & 15, a.d.n_blocks, a.d.Hkv, 16, D);
#pragma unroll 1
            for (int i = ch0; i < ch1; ++i) {
              const float z = __half2float(at[i]);
              if (isfinite(z)) continue;
              if (final) tree_store(a.out, a.out_type, off + i, tree_load(a.out, a.out_type, off + i) + z);
              else rec[((i / 4) * kR + row_in) * 4 + (i & 3)] += z;
            }
          }
        }
        if (!final && valid && (kWide || b == 0)) {
          rec[kR * D + row_in] = M;
          rec[kR * D + kR + row_in] = L;
        }
        tc_fence_before();
      }
      if (in) {
        mbar_arrive(&oempty[kWide ? b : 0]);  // O may be written again
        ++units;
      }
      if (t0 > 0 && cut.awaited)  // a part for another CTA (a group that sat out has nothing of it)
        asm volatile("bar.arrive 4, 288;" ::: "memory");
      left -= t1 - t0;
      tile = 0;
      u = nu;
    }
  }

  __syncthreads();
  // the last commit has arrived (every MMA and every commit before it has); after an abort also the copies in flight
  const uint64_t w0 = global_ns();
  if (warp == 9)
    while (!mbar_try(mma_done, 0) && global_ns() - w0 < kWaitLimitNs) {
    }
  if (threadIdx.x == 256 && *abort_flag)
    for (int i = max(flags[2] - kS, 0); i < flags[2]; ++i)
      while (!mbar_try(&full[i % kS], (i / kS) & 1) && global_ns() - w0 < kWaitLimitNs) {
      }
  __syncthreads();
  if (threadIdx.x < cut.follow) tree_retire(a.m, here + (threadIdx.x + 1) * cut.step);
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

template <int D, bool kWide, int kKind>
cudaError_t one(const TreeAttendArgs& a, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  static SmemOptIn opt;
  constexpr bool kQ8 = kKind != kTreeF16;
  constexpr int smem = TcSmem<D, kQ8>::kBytes;
  static_assert(smem <= 232448, "one CTA per SM");
  cudaError_t e = opt.ensure(k_tree_attend_tc<D, kWide, kKind>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_attend_tc<D, kWide, kKind>, ctas, kQ8 ? kTcTreeThreadsQ8 : kTcTreeThreads, smem, s, *tm, a);
}
template <int D, bool kWide>
cudaError_t kinds(const TreeAttendArgs& a, int kv_type, const CUtensorMap* tm, int ctas, cudaStream_t s) {
  return kv_type == kTreeF16    ? one<D, kWide, kTreeF16>(a, tm, ctas, s)
         : kv_type == kTreeE4m3 ? one<D, kWide, kTreeE4m3>(a, tm, ctas, s)
                                : one<D, kWide, kTreeI8>(a, tm, ctas, s);
}

}  // namespace

cudaError_t launch_tree_attend_tc(const TreeAttendArgs& a, int kv_type, const CUtensorMap* tm, int ctas, bool wide, cudaStream_t s) {
  switch (a.d.D) {
    case 64: return wide ? kinds<64, true>(a, kv_type, tm, ctas, s) : kinds<64, false>(a, kv_type, tm, ctas, s);
    case 128: return wide ? kinds<128, true>(a, kv_type, tm, ctas, s) : kinds<128, false>(a, kv_type, tm, ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dec
