// tree.cu - draft trees over the paged KV cache through the C ABI: the plan of
// a step's trees (validated on the host, one upload), the rotary tables, and
// the entry points of append, attention and commit.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <vector>

#include "../../include/dec.h"
#include "internal.h"
#include "tree.h"

using namespace dec;

namespace {

constexpr int kStages = 4;  // pinned upload buffers in flight
constexpr int kTreeMaxTokens = 1 << 20;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(code, buf);
}

#define TREE_CUDA(call)                                                                 \
  do {                                                                                  \
    cudaError_t e_ = (call);                                                            \
    if (e_ != cudaSuccess) return fail(DEC_ECUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: error word | the plan's upload | attention records.
struct TreeLayout {
  size_t meta, part, total;
  size_t meta_ints;
};

// Which attention kernel takes a batch whose widest sequence has max_rows rows
// (nodes x query heads per KV head).  Measured at 32 sequences over 1024-2048
// keys, 16:8 heads x 128: 16 rows 38.4 us on mma.sync against 46 on tcgen05; 32
// rows 83 (its accumulators spill at two row tiles a warp) against 51; at 8
// sequences over 8000 keys with 512 rows, narrow units 211 us, wide ones 114.
TreeVariant variant_for(int kv_type, int D, int max_rows) {
  if (kv_type == kTreeF32) return {kTreeFfma, max_rows <= 16 ? 16 : 32, 64, D == 128 ? 2 : 3, 2, 0};
  // a unit's start and end in tiles of 8-bit keys: 2 (8 x 256 over 8000, e4m3: 130.8 us, with 1 131.7, with 4 133.3, with 6
  // 139.3; 32 x 64, i8, over 1024-2048 52.6, with 4 53.3, over 3000 79.3, 82.5; over one length of 1500 54.5, 52.5)
  const int unit = kv_type == kTreeF16 ? 4 : 2;
  if (D >= 64 && max_rows > 128) return {kTreeTcWide, 256, 128, 1, unit, 50};
  if (D >= 64 && max_rows > 16) return {kTreeTc, 128, 128, 1, unit, 25};
  // Three CTAs per SM fill the GPU while the kernel before still drains: of 456 the last ones found no place until others had
  // ended, 12 us later.  With 0, 2, 4, 8, 16 places left free 32 x 1 over 1500 takes 27.5, 23.9, 23.2, 23.1, 23.4 us, over
  // 6000 81.2, 69.6, 66.4, 66.3, 66.2, 64 x 1 over 1500 46.1, 40.7, 38.7, 37.8, 39.0.  Two CTAs per SM leave registers for a
  // third and wait for nothing: 32 x 8 over 1500 31.3 us with every place, 31.8 with 4 fewer, 31.7 with 8
  if (kv_type != kTreeF16) return max_rows > 8 && D == 128 ? TreeVariant{kTreeMmaQ8, 16, 64, 2, 2, 0, 0} : TreeVariant{kTreeMmaQ8, max_rows > 8 ? 16 : 8, 64, 3, 2, 0, 8};
  return {kTreeMma, max_rows <= 16 ? 16 : 32, 64, 2, 2, 0};
}
// The rows of a sequence walk the keys side by side in the wide kernel alone, a CTA for each of its row tiles.
constexpr int kWideGang = 4;
static_assert(kTreeMaxNodes * 4 <= kWideGang * 256, "at most four query heads per KV head");
// Records of the attention kernels: two per CTA; rows of all of them, per SM.
constexpr int kRecordRows = 2 * 256;

TreeLayout tree_layout(const dec_config& c, bool q8, int max_seqs, int max_tokens, int max_blocks, int sms) {
  TreeLayout L{};
  const size_t S = max_seqs, N = max_tokens, P = (size_t)sms * kTreeMaxCtasPerSm;
  // header, flags, seq_start, seqs, pos, dst, parents, mask, cuts, merges, reads, pages (a node at least in each), tables
  // (each piece 16-byte aligned)
  L.meta_ints = kHdrInts + P + (S + 1) + 4 * S + 3 * N + N * (kTreeMaxNodes / 32) + P * 20 + 8 * (S + 1) + (q8 ? 4 * N : 0) + S * (size_t)max_blocks + 16 * 4;
  L.meta = 256;
  L.part = up256(L.meta + L.meta_ints * 4);
  L.total = up256(L.part + (size_t)sms * kRecordRows * (size_t)(c.head_dim + 2) * 4);
  return L;
}

// The device a plan belongs to is current while a call runs.
struct DeviceGuard {
  int was = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    int cur = 0;
    ok = cudaGetDevice(&cur) == cudaSuccess;
    if (ok && cur != dev) {
      ok = cudaSetDevice(dev) == cudaSuccess;
      was = cur;
    }
  }
  ~DeviceGuard() {
    if (was >= 0) cudaSetDevice(was);
  }
};

int type_bytes(int t) { return t == kTreeF32 ? 4 : 2; }
bool type_ok(int t) { return t == kTreeF32 || t == kTreeF16 || t == kTreeBf16; }

}  // namespace

struct dec_tree {
  const dec_pool* pool;  // its block bookkeeping, read by dec_tree_set alone
  void* slabs;           // what the kernels need of the pool
  int n_blocks;
  dec_config cfg;
  int device, sms, max_seqs, max_tokens, max_blocks;
  char* ws;
  TreeLayout lay;
  int32_t* stage[kStages];
  cudaEvent_t stage_ev[kStages];
  int stage_next;
  bool f16, q8;  // f16: computed on the f16 tensor cores (f16 and 8-bit caches)
  int kv_type;
  float* scales;  // of an 8-bit cache
  CUtensorMap tm, tm_groups;  // boxes of a block: K and V row by row, and K or V by groups of eight rows
  bool cleared;               // the error word has been
  // the plan that was set last
  bool set;
  TreeMeta meta;
  int kernel, max_nodes, max_position, ctas, n_merges, max_parts, n_pages, read_blocks[2];
  int64_t read_rows[2];
};

namespace {

// The pool's tensor maps for the f16 attention, in 128-byte (64-byte for
// head_dim 32) swizzled rows.  [64 channels][rows of a slab][halves of the
// head][K, V][layer and block]: one box is the K and V of one KV head of one
// block.  groups: [64 channels][8 rows][halves][groups of 8 rows][layer, block,
// K or V]: one box is the K or the V of one KV head of one block, the halves of
// eight rows next to each other, so that the groups of a tile of many blocks
// lie evenly apart, as the tensor cores want them.  8-bit codes: a box as the
// first, rows of the whole head (128, 64 or 32 bytes, swizzled as wide).
bool pool_map(CUtensorMap* out, const dec_pool* p, bool groups) {
  typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(f);
    return nullptr;
  }();
  if (!fn) return false;
  const dec_config& c = p->cfg;
  const cuuint64_t D = c.head_dim, bd = D >= 64 ? 64 : D, slab = (cuuint64_t)c.n_kv_heads * 16 * D * 2;
  const cuuint64_t n = (cuuint64_t)c.n_layers * p->n_blocks, h = D / bd;
  cuuint64_t dims[5] = {bd, (cuuint64_t)c.n_kv_heads * 16, h, 2, n};
  cuuint64_t strides[4] = {D * 2, bd * 2, slab, 2 * slab};
  cuuint32_t box[5] = {(cuuint32_t)bd, 16, (cuuint32_t)h, 2, 1};
  if (groups) {
    dims[1] = 8, dims[3] = (cuuint64_t)c.n_kv_heads * 2, dims[4] = 2 * n;
    strides[2] = 8 * D * 2, strides[3] = slab;
    box[1] = 8;
  }
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  if (pool_q8(p)) {
    const cuuint64_t codes = (cuuint64_t)c.n_kv_heads * 16 * D, d8[4] = {D, (cuuint64_t)c.n_kv_heads * 16, 2, n}, s8[3] = {D, codes, 2 * codes};
    const cuuint32_t b8[4] = {(cuuint32_t)D, 16, 2, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p->slabs, d8, s8, b8, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              D == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
              : D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                        : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  return fn(out, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, p->slabs, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            bd == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Every check of a batch of trees, host data only.
int check_trees(const dec_pool* pool, const dec_tree_batch* b) {
  if (!pool || !b) return fail(DEC_EINVAL, "NULL argument");
  const dec_config& c = pool->cfg;
  const int S = b->n_seqs, N = b->n_tokens, B = c.block_tokens;
  if (S < 1 || N < 1) return fail(DEC_EINVAL, "empty step: %d sequences, %d nodes", S, N);
  if (!b->seq_start || !b->ctx || !b->block_table) return fail(DEC_EINVAL, "NULL batch array");
  if (b->max_blocks < 1) return fail(DEC_EINVAL, "max_blocks must be at least 1");
  if (b->seq_start[0] != 0 || b->seq_start[S] != N) return fail(DEC_EINVAL, "seq_start must run from 0 to n_tokens");
  for (int s = 0; s < S; ++s)  // before any array is indexed by it
    if (b->seq_start[s + 1] < b->seq_start[s]) return fail(DEC_EINVAL, "seq_start decreases at sequence %d", s);
  std::vector<int32_t> written, depth;
  for (int s = 0; s < S; ++s) {
    const int a0 = b->seq_start[s], T = b->seq_start[s + 1] - a0, ctx = b->ctx[s];
    if (T > kTreeMaxNodes) return fail(DEC_ERANGE, "sequence %d has %d nodes, more than %d", s, T, kTreeMaxNodes);
    if (ctx < 0 || ctx > c.max_positions) return fail(DEC_ERANGE, "context of sequence %d outside 0 .. max_positions", s);
    if (T == 0) continue;
    depth.assign(T, 0);
    for (int i = 0; i < T; ++i) {
      const int p = b->parents ? b->parents[a0 + i] : i - 1;
      if (p == DEC_TREE_PAD) {
        depth[i] = -1;
        continue;
      }
      if (p < -1 || p >= i) return fail(DEC_EINVAL, "node %d of sequence %d: parent %d is not an earlier node", i, s, p);
      if (p >= 0 && depth[p] < 0) return fail(DEC_EINVAL, "node %d of sequence %d: its parent is padding", i, s);
      depth[i] = p < 0 ? 0 : depth[p] + 1;
      if (ctx + depth[i] >= c.max_positions)
        return fail(DEC_ERANGE, "position %d past the context (%d)", ctx + depth[i], c.max_positions);
    }
    const int nb = (ctx + T - 1) / B + 1;
    if (nb > b->max_blocks) return fail(DEC_ERANGE, "block table of sequence %d too short for slot %d", s, ctx + T - 1);
    for (int i = 0; i < nb; ++i) {
      const int id = b->block_table[(size_t)s * b->max_blocks + i];
      if (id < 0 || id >= pool->n_blocks || pool->refs[id] <= 0)
        return fail(DEC_EBLOCK, "sequence %d names block %d which is not allocated", s, id);
      if (i >= ctx / B) {  // nodes' K/V go there
        if (pool->refs[id] != 1 || pool->registered[id])
          return fail(DEC_EBLOCK, "sequence %d would write block %d, which is shared (refcount %d) or in the prefix cache",
                      s, id, pool->refs[id]);
        written.push_back(id);
      }
    }
  }
  std::sort(written.begin(), written.end());
  const auto dup = std::adjacent_find(written.begin(), written.end());
  if (dup != written.end()) return fail(DEC_EBLOCK, "block %d would be written for two slots of the step", *dup);
  return DEC_OK;
}

// Distribute the attention work over `grid` CTAs: cuts, and the units that CTAs
// share.  Sequences fall into classes of equally many row tiles; a class gets
// CTAs by its share of the work, in gangs of one CTA per row tile (up to
// `max_gang`) that walk the same keys at the same time, so that a tile's
// second reader finds it in L2.  The gangs of a class cut its (sequence, head)
// list into equal runs, a unit's start and end counted as unit_cost tiles.
// Returns the merges, of up to *parts, that a second kernel is needed for: none
// where the CTAs that start shared units join the others' parts (cuts' follow).
int distribute(const dec_config& c, std::vector<TreeSeq>& seqs, const TreeVariant& var, int grid, int max_gang, TreeCut* cut,
               TreeMerge* mrg, int* parts) {
  const int G = c.n_heads / c.n_kv_heads, R = var.row_tile, K = var.tile_keys, Hkv = c.n_kv_heads;
  auto row_tiles = [&](const TreeSeq& s) { return (s.nodes * G + R - 1) / R; };
  auto tiles = [&](const TreeSeq& s) { return (s.ctx + s.nodes + K - 1) / K; };
  auto gang = [&](const TreeSeq& s) { return std::min(row_tiles(s), max_gang); };
  std::stable_sort(seqs.begin(), seqs.end(), [&](const TreeSeq& x, const TreeSeq& y) { return gang(x) < gang(y); });
  // work of each class, and its CTAs: whole gangs, one at least, the rest to whichever class is most behind
  std::vector<double> work(max_gang + 1, 0.0);
  std::vector<int> gangs(max_gang + 1, 0);
  for (const TreeSeq& s : seqs) work[gang(s)] += (double)Hkv * row_tiles(s) * (tiles(s) + var.unit_cost);
  int left = grid;
  for (int g = 1; g <= max_gang; ++g)
    if (work[g] > 0) {
      gangs[g] = 1;
      left -= g;
    }
  while (true) {
    int most = 0;
    for (int g = 1; g <= max_gang; ++g)
      if (work[g] > 0 && g <= left && (!most || work[g] / (gangs[g] * g) > work[most] / (gangs[most] * most))) most = g;
    if (!most) break;
    ++gangs[most];
    left -= most;
  }
  int n_mrg = 0, cta = 0;
  for (size_t q0 = 0; q0 < seqs.size();) {
    const int g = gang(seqs[q0]);
    size_t q1 = q0;
    while (q1 < seqs.size() && gang(seqs[q1]) == g) ++q1;
    // the class as a line of units: (sequence, head, row tile) for a gang of one, (sequence, head) for a larger one, whose
    // members have a row tile each (a gang is as large as its sequences have row tiles, if it may be larger than one)
    struct Unit {
      int q, head, row_tile, tiles;  // the first member's
    };
    std::vector<Unit> units;
    double cost = 0;
    int longest = 0;
    for (size_t q = q0; q < q1; ++q)
      for (int h = 0; h < Hkv; ++h)
        for (int rt = 0; rt < row_tiles(seqs[q]); rt += g) {
          units.push_back({(int)q, h, rt, tiles(seqs[q])});
          cost += tiles(seqs[q]) + var.unit_cost;
          longest = std::max(longest, tiles(seqs[q]));
        }
    // cuts as (unit, tile); near a unit's border the cut moves there, where that costs less than another piece
    const int n = gangs[g];
    const double run = cost / n;
    // short units that all have a gang of their own stay whole: joining parts costs more than up to three tiles one after
    // the other (4 sequences x 64 nodes over 300 keys, three tiles: 11.4 us against 14.3 with cuts from two tiles on; 1 x 5
    // over 180: 6.5 against 6.4; 1 x 64 over 500, five tiles: 13.5 whole, 13.9 cut; four tiles of 64 keys: 9.5 whole, 9.2 cut)
    const bool split = (int)units.size() > n || longest > 3;
    const int snap = (int)std::min(var.unit_cost / 2.0, run / 8);
    std::vector<std::pair<int, int>> at;  // distinct, ascending
    size_t x = 0;
    double before = 0;
    for (int i = 0; i < n; ++i) {
      const double pos = cost * i / n;
      while (x < units.size() && before + units[x].tiles + var.unit_cost <= pos) before += units[x++].tiles + var.unit_cost;
      if (x == units.size()) break;
      int t = std::min((int)(pos - before), units[x].tiles);
      std::pair<int, int> here{(int)x, t};
      if (t <= snap || !split) here.second = 0;
      else if (units[x].tiles - t <= snap) here = {(int)x + 1, 0};
      if (here.first < (int)units.size() && (at.empty() || at.back() < here)) at.push_back(here);
    }
    const int used = (int)at.size();
    at.push_back({(int)units.size(), 0});
    for (int i = 0; i < used; ++i)
      for (int member = 0; member < g; ++member) {
        TreeCut& o = cut[cta + i * g + member];
        o = {};
        for (int y = at[i].first; y <= at[i + 1].first && y < (int)units.size(); ++y) {
          const Unit& w = units[y];
          const int t0 = y == at[i].first ? at[i].second : 0, t1 = y == at[i + 1].first ? at[i + 1].second : w.tiles;
          if (t1 <= t0) continue;
          if (o.count == 0) o = {w.q, w.head, w.row_tile + member, t0, 0, g, 0, 0, seqs[w.q]};
          o.count += t1 - t0;
        }
      }
    // units with a cut inside
    for (int i = 1; i < used; ++i) {
      if (at[i].second == 0 || (i > 1 && at[i - 1].first == at[i].first && at[i - 1].second > 0)) continue;
      const Unit& w = units[at[i].first];
      int last = i;
      while (last + 1 < used && at[last + 1].first == at[i].first) ++last;
      for (int member = 0; member < g; ++member) {
        mrg[n_mrg++] = {w.head, w.row_tile + member, cta + (i - 1) * g + member, cta + last * g + member, g, seqs[w.q].node0, seqs[w.q].nodes, 0};
      }
    }
    cta += used * g;
    q0 = q1;
  }
  // the first blocks take the last places: none without work before one that has some
  const int idle = grid - cta;
  std::copy_backward(cut, cut + cta, cut + grid);
  std::fill(cut, cut + idle, TreeCut{});
  for (int i = 0; i < n_mrg; ++i) {
    mrg[i].c0 += idle;
    mrg[i].c1 += idle;
  }
  // Joining costs a flag's round trip and the reads behind it at the end of the call, a second kernel its launch and the
  // records of all shared units.  The tcgen05 kernels' large records are better joined, once enough units are shared
  // (joined, second kernel: 32 x 64 over 1024-2048 51.9 us, 56.4; 16 x 64 over 2000 35.9, 40.5; 8 x 64 over 2000 29.1, 29.4;
  // wide: 8 x 256 over 8000 114, 119; 5 x 256 over 4000, 53 units per hundred CTAs, 57.3, 59.2; 4 x 256 there, 42 per
  // hundred, 51.0, 50.6; 8 x 128 over 1000, 42 per hundred, 34.0, 30.4).  The small ones of 16 rows are not (mma.sync: 32 x
  // 8 over 1024-2048 39.4, 38.7; 64 x 4 over 500-1500 49.2, 47.8; 24 x 8 over 3000-4000 60.5, 58.5).  An fp32 cache has it
  // either way (16 x 4 over 1000-1400 108.6, 106.2; 40 x 8 over 300-600 102.8, 104.8) and does without.
  bool join = var.join > 0 && n_mrg * 100 >= grid * var.join;
  *parts = 0;
  for (int i = 0; i < n_mrg; ++i) {
    *parts = std::max(*parts, (mrg[i].c1 - mrg[i].c0) / mrg[i].stride + 1);
    if (*parts > 3) join = false;
  }
  if (!join) return n_mrg;
  for (int i = 0; i < n_mrg; ++i) {
    cut[mrg[i].c0].follow = (mrg[i].c1 - mrg[i].c0) / mrg[i].stride;
    for (int c = mrg[i].c0 + mrg[i].stride; c <= mrg[i].c1; c += mrg[i].stride) cut[c].awaited = 1;
  }
  return 0;
}

// Fill the pinned image of the plan and the kernels' view of its upload;
// returns the ints used.
size_t build_plan(dec_tree* t, const dec_tree_batch* b, int32_t* H) {
  const dec_config& c = t->cfg;
  const int S = b->n_seqs, N = b->n_tokens, G = c.n_heads / c.n_kv_heads;
  size_t o = 0;
  auto take = [&](size_t n) { size_t at = o; o = (o + n + 3) & ~size_t(3); return at; };
  int max_nodes = 0, max_position = 0;
  for (int s = 0; s < S; ++s) max_nodes = std::max(max_nodes, b->seq_start[s + 1] - b->seq_start[s]);
  const int W = std::max((max_nodes + 31) / 32, 1);
  const TreeVariant var = variant_for(t->kv_type, c.head_dim, max_nodes * G);
  const int grid = std::max(t->sms * var.ctas_per_sm - var.spare, t->sms);
  // Where a piece lies depends on S, N and W alone, which a captured call is replayed with: the cuts and merges have room for
  // any variant's grid, as append, commit and reading back follow plans whose attention takes another one.
  const size_t P = (size_t)t->sms * kTreeMaxCtasPerSm;
  const size_t h_hdr = take(kHdrInts), h_flags = take(P), h_start = take(S + 1), h_seqs = take((size_t)S * 4), h_pos = take(N), h_dst = take(N),
               h_par = take(N), h_anc = take((size_t)N * W), h_cut = take(P * 12), h_mrg = take(P * 8),
               h_reads = take((size_t)(S + 1) * 8), h_pages = take(t->q8 ? (size_t)N * 4 : 0), h_tables = o;
  std::vector<TreeSeq> seqs;
  TreePage* pages = reinterpret_cast<TreePage*>(H + h_pages);
  TreeReadSeq read{};
  int64_t read_rows[2] = {0, 0};  // sequences may share their cached blocks: more rows than the pool has slots
  int n_pages = 0;
  for (int s = 0; s < S; ++s) {
    const int a0 = b->seq_start[s], T = b->seq_start[s + 1] - a0, ctx = b->ctx[s];
    H[h_start + s] = a0;
    read.tab = (int32_t)(o - h_tables);
    read.ctx = ctx;
    read.nodes = T;
    for (int i = 0; i < 2; ++i) read.rows[i] = (int32_t)std::min<int64_t>(read_rows[i], INT32_MAX);
    reinterpret_cast<TreeReadSeq*>(H + h_reads)[s] = read;
    if (T == 0) continue;
    read.blocks[0] += (ctx + T + 15) / 16;
    read.blocks[1] += (ctx + T + 15) / 16 - ctx / 16;
    read_rows[0] += ctx + T;
    read_rows[1] += ctx % 16 + T;
    seqs.push_back({a0, T, ctx, (int32_t)(o - h_tables)});
    const int32_t* row = b->block_table + (size_t)s * b->max_blocks;
    const int nb = (ctx + T + 15) / 16;
    std::copy(row, row + nb, H + o);
    o += nb;
    for (int i = 0; t->q8 && i < T;) {
      const int slot = (ctx + i) & 15, in = std::min(T - i, 16 - slot);
      pages[n_pages++] = {row[(ctx + i) >> 4], a0 + i, slot, in};
      i += in;
    }
    uint32_t* anc = reinterpret_cast<uint32_t*>(H + h_anc + (size_t)a0 * W);
    for (int i = 0; i < T; ++i) {
      const int p = b->parents ? b->parents[a0 + i] : i - 1;
      uint32_t* w = anc + (size_t)i * W;
      H[h_par + a0 + i] = p;
      H[h_dst + a0 + i] = row[(ctx + i) >> 4] * 16 + ((ctx + i) & 15);  // an accepted node may move to a padding node's slot
      if (p == DEC_TREE_PAD) {
        std::fill(w, w + W, 0u);
        H[h_pos + a0 + i] = -1;
        continue;
      }
      if (p < 0) std::fill(w, w + W, 0u);
      else std::copy(anc + (size_t)p * W, anc + (size_t)(p + 1) * W, w);
      w[i >> 5] |= 1u << (i & 31);
      H[h_pos + a0 + i] = p < 0 ? ctx : H[h_pos + a0 + p] + 1;
      max_position = std::max(max_position, H[h_pos + a0 + i]);
    }
  }
  H[h_start + S] = N;
  reinterpret_cast<TreeReadSeq*>(H + h_reads)[S] = read;
  static_assert(sizeof(TreeSeq) == 16 && sizeof(TreeCut) == 48 && sizeof(TreeMerge) == 32 && sizeof(TreePage) == 16 && sizeof(TreeReadSeq) == 32, "as the pieces are measured above");
  const int n_mrg = distribute(c, seqs, var, grid, var.kernel == kTreeTcWide ? kWideGang : 1, reinterpret_cast<TreeCut*>(H + h_cut),
                               reinterpret_cast<TreeMerge*>(H + h_mrg), &t->max_parts);
  std::fill(H + h_flags, H + h_flags + P, 0);
  std::copy(seqs.begin(), seqs.end(), reinterpret_cast<TreeSeq*>(H + h_seqs));
  std::fill(H + h_hdr, H + h_hdr + kHdrInts, 0);
  H[h_hdr + kHdrSeqs] = S;
  H[h_hdr + kHdrTokens] = N;
  H[h_hdr + kHdrWords] = W;
  H[h_hdr + kHdrRowTile] = var.row_tile;
  H[h_hdr + kHdrMerges] = n_mrg;
  H[h_hdr + kHdrPages] = n_pages;
  for (int i = 0; i < 2; ++i) H[h_hdr + kHdrRows + i] = read_rows[i] > INT32_MAX ? -1 : (int32_t)read_rows[i];  // -1: no call's number
  int32_t* d = reinterpret_cast<int32_t*>(t->ws + t->lay.meta);
  TreeMeta& m = t->meta;
  m.hdr = d + h_hdr;
  m.seq_start = d + h_start;
  m.seqs = reinterpret_cast<const TreeSeq*>(d + h_seqs);
  m.pos = d + h_pos;
  m.dst = d + h_dst;
  m.parents = d + h_par;
  m.anc = reinterpret_cast<const uint32_t*>(d + h_anc);
  m.cuts = reinterpret_cast<const TreeCut*>(d + h_cut);
  m.merges = reinterpret_cast<const TreeMerge*>(d + h_mrg);
  m.pages = reinterpret_cast<const TreePage*>(d + h_pages);
  m.reads = reinterpret_cast<const TreeReadSeq*>(d + h_reads);
  m.tables = d + h_tables;
  m.err = reinterpret_cast<uint32_t*>(t->ws);
  m.flags = reinterpret_cast<uint32_t*>(d + h_flags);
  m.S = S;
  m.N = N;
  m.words = W;
  m.row_tile = var.row_tile;
  m.tile_keys = var.tile_keys;
  t->kernel = var.kernel;
  t->max_nodes = max_nodes;
  t->max_position = max_position;
  t->ctas = grid;
  t->n_merges = n_mrg;
  t->n_pages = n_pages;
  for (int i = 0; i < 2; ++i) {
    t->read_blocks[i] = read.blocks[i];
    t->read_rows[i] = read_rows[i];
  }
  return o;
}

TreePoolDims pool_dims(const dec_tree* t) {
  const dec_config& c = t->cfg;
  const int G = c.n_heads / c.n_kv_heads;
  return {c.n_heads, c.n_kv_heads, c.head_dim, c.n_layers, t->n_blocks, G == 4 ? 2 : G - 1, (float)c.rms_eps};
}

int check_rope(const dec_rope* r) {
  if (!r) return fail(DEC_EINVAL, "NULL argument");
  if (r->rot_dim < 8 || r->rot_dim > 2 * kRopeMaxPairs || r->rot_dim % 8)
    return fail(DEC_EINVAL, "rot_dim must be a multiple of 8 from 8 to %d", 2 * kRopeMaxPairs);
  if (r->layout != DEC_ROPE_HALF && r->layout != DEC_ROPE_INTERLEAVED) return fail(DEC_EINVAL, "unknown rotary layout");
  if (!(r->base > 1.0) || !std::isfinite(r->base)) return fail(DEC_EINVAL, "rope base must be > 1");
  if (!(r->attn_factor > 0.0) || !std::isfinite(r->attn_factor)) return fail(DEC_EINVAL, "attn_factor must be > 0");
  if (r->scaling == DEC_ROPE_PLAIN) return DEC_OK;
  if (r->scaling != DEC_ROPE_LINEAR && r->scaling != DEC_ROPE_YARN && r->scaling != DEC_ROPE_BANDS)
    return fail(DEC_EINVAL, "unknown rotary scaling");
  if (!(r->factor >= 1.0) || !std::isfinite(r->factor)) return fail(DEC_EINVAL, "scaling factor must be >= 1");
  if (r->scaling == DEC_ROPE_LINEAR) return DEC_OK;
  if (r->orig_positions < 1) return fail(DEC_EINVAL, "orig_positions must be at least 1");
  if (!(r->low > 0.0) || !(r->high > r->low) || !std::isfinite(r->high))
    return fail(DEC_EINVAL, "need 0 < low < high");
  return DEC_OK;
}

// Frequencies of the rotary pairs, in 64 bits (formulas at dec_rope).
void rope_frequencies(const dec_rope& r, double* f) {
  const double two_pi = 6.283185307179586476925;
  const int n = r.rot_dim / 2;
  for (int j = 0; j < n; ++j) f[j] = std::pow(r.base, -2.0 * j / r.rot_dim);
  if (r.scaling == DEC_ROPE_LINEAR) {
    for (int j = 0; j < n; ++j) f[j] /= r.factor;
  } else if (r.scaling == DEC_ROPE_YARN) {
    auto pair_of = [&](double turns) { return r.rot_dim * std::log(r.orig_positions / (turns * two_pi)) / (2.0 * std::log(r.base)); };
    const double lo = std::max(std::floor(pair_of(r.high)), 0.0);
    const double hi = std::min(std::ceil(pair_of(r.low)), (double)(r.rot_dim - 1));
    for (int j = 0; j < n; ++j) {
      const double g = std::min(std::max((j - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      f[j] = f[j] * (1.0 - g) + f[j] / r.factor * g;
    }
  } else if (r.scaling == DEC_ROPE_BANDS) {
    for (int j = 0; j < n; ++j) {
      const double turns = r.orig_positions * f[j] / two_pi;
      const double g = std::min(std::max((turns - r.low) / (r.high - r.low), 0.0), 1.0);
      f[j] = f[j] * g + f[j] / r.factor * (1.0 - g);
    }
  }
}

// Rows of `heads` heads of D elements each, `ld` elements apart, are addressable in 4-element pieces.
int check_rows(const void* p, int64_t ld, int heads, int D, int type, const char* what) {
  if (!type_ok(type)) return fail(DEC_EINVAL, "%s: unknown element type %d", what, type);
  if (ld < (int64_t)heads * D) return fail(DEC_EINVAL, "%s: rows of %d elements overlap at a stride of %lld", what, heads * D, (long long)ld);
  if (((uintptr_t)p & (4 * type_bytes(type) - 1)) || ld % 4)
    return fail(DEC_EINVAL, "%s must be aligned to 4 elements, its row stride a multiple of 4", what);
  return DEC_OK;
}

int check_ready(const dec_tree* t, int layer) {
  if (!t) return fail(DEC_EINVAL, "NULL argument");
  if (!t->set) return fail(DEC_EINVAL, "no trees: dec_tree_set has not been called");
  if (layer < 0 || layer >= t->cfg.n_layers) return fail(DEC_EINVAL, "layer outside the model");
  return DEC_OK;
}

}  // namespace

extern "C" {

int dec_rope_table_bytes(const dec_rope* r, int32_t n_positions, size_t* bytes) {
  int rc = check_rope(r);
  if (rc) return rc;
  if (!bytes) return fail(DEC_EINVAL, "NULL argument");
  if (n_positions < 1 || n_positions > kMaxPositions) return fail(DEC_ERANGE, "n_positions must lie in 1 .. %d", kMaxPositions);
  *bytes = (size_t)n_positions * r->rot_dim * 4;
  return DEC_OK;
}

int dec_rope_table(const dec_rope* r, int32_t n_positions, float* table, size_t bytes, void* stream) {
  size_t need = 0;
  int rc = dec_rope_table_bytes(r, n_positions, &need);
  if (rc) return rc;
  if (!table || ((uintptr_t)table & 15)) return fail(DEC_EINVAL, "table must be 16-byte aligned device memory");
  if (bytes < need) return fail(DEC_EINVAL, "table too small: %zu < %zu", bytes, need);
  RopeTableArgs a{};
  a.table = table;
  a.positions = n_positions;
  a.pairs = r->rot_dim / 2;
  a.mult = r->attn_factor;
  rope_frequencies(*r, a.freq);
  TREE_CUDA(launch_rope_table(a, (cudaStream_t)stream));
  return DEC_OK;
}

int dec_tree_check(const dec_pool* pool, const dec_tree_batch* b) {
  try {
    return check_trees(pool, b);
  } catch (const std::bad_alloc&) {
    return fail(DEC_ECAPACITY, "out of host memory");
  }
}

int dec_tree_workspace_bytes(const dec_pool* pool, int32_t max_seqs, int32_t max_tokens, int32_t max_blocks,
                             size_t* bytes) {
  if (!pool || !bytes) return fail(DEC_EINVAL, "NULL argument");
  if (max_seqs < 1 || max_tokens < 1 || max_blocks < 1) return fail(DEC_EINVAL, "capacities must be at least 1");
  if (max_tokens > kTreeMaxTokens || max_seqs > kTreeMaxTokens || (int64_t)max_seqs * max_blocks > (1 << 28))
    return fail(DEC_ERANGE, "capacities too large");
  int dev = 0, sms = 0;
  TREE_CUDA(cudaGetDevice(&dev));
  TREE_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  *bytes = tree_layout(pool->cfg, pool_q8(pool), max_seqs, max_tokens, max_blocks, sms).total;
  return DEC_OK;
}

void dec_tree_destroy(dec_tree* t) {
  if (!t) return;
  DeviceGuard g(t->device);
  for (int i = 0; i < kStages; ++i) {
    if (t->stage_ev[i]) {
      cudaEventSynchronize(t->stage_ev[i]);  // an upload may still read the pinned buffer
      cudaEventDestroy(t->stage_ev[i]);
    }
    if (t->stage[i]) cudaFreeHost(t->stage[i]);
  }
  delete t;
}

int dec_tree_create(const dec_pool* pool, int32_t max_seqs, int32_t max_tokens, int32_t max_blocks, void* workspace,
                    size_t bytes, dec_tree** out) {
  if (!out) return fail(DEC_EINVAL, "NULL argument");
  size_t need = 0;
  int rc = dec_tree_workspace_bytes(pool, max_seqs, max_tokens, max_blocks, &need);
  if (rc) return rc;
  if (!workspace || ((uintptr_t)workspace & 255)) return fail(DEC_EINVAL, "workspace must be 256-byte aligned device memory");
  if (bytes < need) return fail(DEC_EINVAL, "workspace too small: %zu < %zu", bytes, need);
  dec_tree* t = new (std::nothrow) dec_tree();
  if (!t) return fail(DEC_ECAPACITY, "out of host memory");
  t->pool = pool;
  t->slabs = pool->slabs;
  t->n_blocks = pool->n_blocks;
  t->cfg = pool->cfg;
  t->max_seqs = max_seqs;
  t->max_tokens = max_tokens;
  t->max_blocks = max_blocks;
  t->ws = (char*)workspace;
  t->f16 = pool->cfg.mode != DEC_FP32;
  t->q8 = pool_q8(pool);
  t->kv_type = pool->kv_type;
  t->scales = t->q8 ? reinterpret_cast<float*>(reinterpret_cast<char*>(pool->slabs) + pool->scales) : nullptr;
  cudaError_t e = cudaGetDevice(&t->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&t->sms, cudaDevAttrMultiProcessorCount, t->device);
  t->lay = tree_layout(t->cfg, t->q8, max_seqs, max_tokens, max_blocks, t->sms);
  for (int i = 0; i < kStages && e == cudaSuccess; ++i) {
    e = cudaMallocHost((void**)&t->stage[i], t->lay.meta_ints * 4);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&t->stage_ev[i], cudaEventDisableTiming);
  }
  if (e != cudaSuccess) {
    rc = fail(DEC_ECUDA, "dec_tree_create: %s", cudaGetErrorString(e));
  } else if (t->f16 && !(pool_map(&t->tm, pool, false) && (t->q8 || pool_map(&t->tm_groups, pool, true)))) {
    rc = fail(DEC_ECUDA, "tensor map of the KV pool failed");
  }
  if (rc) {
    dec_tree_destroy(t);
    return rc;
  }
  *out = t;
  return DEC_OK;
}

int dec_tree_set(dec_tree* t, const dec_tree_batch* b, void* stream) {
  if (!t) return fail(DEC_EINVAL, "NULL argument");
  int rc = dec_tree_check(t->pool, b);
  if (rc) return rc;
  if ((int64_t)b->n_tokens * (t->cfg.n_heads + 2 * t->cfg.n_kv_heads) > INT32_MAX)
    return fail(DEC_ERANGE, "%d nodes of %d heads are too many rows", b->n_tokens, t->cfg.n_heads);
  if (b->n_seqs > t->max_seqs || b->n_tokens > t->max_tokens)
    return fail(DEC_ERANGE, "%d sequences and %d nodes exceed the plan (%d / %d)", b->n_seqs, b->n_tokens, t->max_seqs,
                t->max_tokens);
  for (int s = 0; s < b->n_seqs; ++s) {
    const int T = b->seq_start[s + 1] - b->seq_start[s];
    if (T > 0 && (b->ctx[s] + T + 15) / 16 > t->max_blocks)
      return fail(DEC_ERANGE, "sequence %d needs %d blocks, the plan holds %d", s, (b->ctx[s] + T + 15) / 16, t->max_blocks);
  }
  DeviceGuard g(t->device);
  if (!g.ok) return fail(DEC_ECUDA, "the plan's device cannot be made current");
  cudaStream_t st = (cudaStream_t)stream;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  TREE_CUDA(cudaStreamIsCapturing(st, &cap));
  if (cap != cudaStreamCaptureStatusNone)
    return fail(DEC_EINVAL, "dec_tree_set reads host data and cannot be captured: call it before the captured calls");
  const int slot = t->stage_next;
  TREE_CUDA(cudaEventSynchronize(t->stage_ev[slot]));  // the copy that last used this buffer has run
  t->stage_next = (slot + 1) % kStages;
  t->set = false;
  size_t ints = 0;
  try {
    ints = build_plan(t, b, t->stage[slot]);
  } catch (const std::bad_alloc&) {
    return fail(DEC_ECAPACITY, "out of host memory");
  }
  if (!t->cleared) {  // the error word, once, in the order of the stream that the plan is first used on
    TREE_CUDA(cudaMemsetAsync(t->ws, 0, 256, st));
    t->cleared = true;
  }
  TREE_CUDA(cudaMemcpyAsync(t->ws + t->lay.meta, t->stage[slot], ints * 4, cudaMemcpyHostToDevice, st));
  TREE_CUDA(cudaEventRecord(t->stage_ev[slot], st));
  t->set = true;
  return DEC_OK;
}

int dec_tree_status(dec_tree* t, void* stream, uint32_t* flags) {
  if (!t || !flags) return fail(DEC_EINVAL, "NULL argument");
  DeviceGuard g(t->device);
  if (!g.ok) return fail(DEC_ECUDA, "the plan's device cannot be made current");
  cudaStream_t st = (cudaStream_t)stream;
  uint32_t v = 0;
  if (t->cleared) {  // else no call has been made
    TREE_CUDA(cudaMemcpyAsync(&v, t->ws, 4, cudaMemcpyDeviceToHost, st));
    TREE_CUDA(cudaMemsetAsync(t->ws, 0, 4, st));
  }
  TREE_CUDA(cudaStreamSynchronize(st));
  *flags = v;
  return DEC_OK;
}

int dec_debug_tree_join(dec_tree* t, int32_t late, uint64_t limit_ns, int32_t* left, void* stream) {
  int rc = check_ready(t, 0);
  if (rc) return rc;
  if (!left) return fail(DEC_EINVAL, "NULL argument");
  if (limit_ns < 1000 || limit_ns > 1000000000ull) return fail(DEC_EINVAL, "the test limit must lie between 1 us and 1 s");
  DeviceGuard g(t->device);
  if (!g.ok) return fail(DEC_ECUDA, "the plan's device cannot be made current");
  cudaStream_t st = (cudaStream_t)stream;
  TREE_CUDA(launch_tree_join_test(t->meta, late, limit_ns, st));
  int32_t v = 0;
  TREE_CUDA(cudaMemcpyAsync(&v, t->meta.flags, 4, cudaMemcpyDeviceToHost, st));
  TREE_CUDA(cudaStreamSynchronize(st));
  *left = v;
  return DEC_OK;
}

int dec_tree_append(dec_tree* t, int32_t layer, const dec_tree_qkv* x, void* stream) {
  int rc = check_ready(t, layer);
  if (rc) return rc;
  if (!x) return fail(DEC_EINVAL, "NULL argument");
  const dec_config& c = t->cfg;
  const int D = c.head_dim;
  if (!x->k != !x->v) return fail(DEC_EINVAL, "keys and values come together");
  if (!x->q && !x->k) return fail(DEC_EINVAL, "neither queries nor keys");
  if (x->q && !x->q_out) return fail(DEC_EINVAL, "q_out is NULL");
  if (x->q) {
    if ((rc = check_rows(x->q, x->ldq, c.n_heads, D, x->in_type, "q"))) return rc;
    if ((rc = check_rows(x->q_out, x->ldqo, c.n_heads, D, x->q_type, "q_out"))) return rc;
    if (x->q_out == x->q && (x->q_type != x->in_type || x->ldqo != x->ldq))
      return fail(DEC_EINVAL, "queries in place need one type and one row stride: other rows are still to be read");
  }
  if (x->k) {
    if ((rc = check_rows(x->k, x->ldk, c.n_kv_heads, D, x->in_type, "k"))) return rc;
    if ((rc = check_rows(x->v, x->ldv, c.n_kv_heads, D, x->in_type, "v"))) return rc;
  }
  if (((uintptr_t)x->q_norm | (uintptr_t)x->k_norm) & 15) return fail(DEC_EINVAL, "gains must be 16-byte aligned");
  TreeAppendArgs a{};
  if (x->rope) {
    if ((rc = check_rope(x->rope))) return rc;
    if (x->rope->rot_dim > D) return fail(DEC_EINVAL, "rot_dim %d above the head's %d channels", x->rope->rot_dim, D);
    if (!x->rope_table || ((uintptr_t)x->rope_table & 15)) return fail(DEC_EINVAL, "rope_table must be a 16-byte aligned dec_rope_table");
    if (x->rope_positions < t->max_position + 1)
      return fail(DEC_ERANGE, "the rotary table holds %d positions, the trees reach %d", x->rope_positions, t->max_position);
    a.rope = x->rope_table;
    a.rot = x->rope->rot_dim;
    a.rope_positions = x->rope_positions;
    a.interleaved = x->rope->layout == DEC_ROPE_INTERLEAVED;
  }
  DeviceGuard g(t->device);
  if (!g.ok) return fail(DEC_ECUDA, "the plan's device cannot be made current");
  a.m = t->meta;
  a.d = pool_dims(t);
  a.q = x->q;
  a.k = x->k;
  a.v = x->v;
  a.ldq = x->ldq;
  a.ldk = x->ldk;
  a.ldv = x->ldv;
  a.ldo = x->ldqo;
  a.q_norm = x->q_norm;
  a.k_norm = x->k_norm;
  a.q_out = x->q_out;
  a.in_type = x->in_type;
  a.q_type = x->q_type;
  a.kv_type = t->kv_type;
  a.scales = t->scales;
  a.n_pages = t->n_pages;
  a.sms = t->sms;
  a.layer = layer;
  a.kv = t->slabs;
  TREE_CUDA(t->q8 ? launch_tree_append_q8(a, (cudaStream_t)stream) : launch_tree_append(a, (cudaStream_t)stream));
  return DEC_OK;
}

int dec_tree_attend(dec_tree* t, int32_t layer, const void* q, int32_t q_type, int64_t ldq, void* out, int32_t out_type,
                    int64_t ldo, void* stream) {
  int rc = check_ready(t, layer);
  if (rc) return rc;
  if (!q || !out) return fail(DEC_EINVAL, "NULL argument");
  const dec_config& c = t->cfg;
  if ((rc = check_rows(q, ldq, c.n_heads, c.head_dim, q_type, "q"))) return rc;
  if ((rc = check_rows(out, ldo, c.n_heads, c.head_dim, out_type, "out"))) return rc;
  if (q == out) return fail(DEC_EINVAL, "the output must not be the queries: other units still read them");
  if (t->f16 && out_type == DEC_T_F32)
    return fail(DEC_EINVAL, "an f16 or 8-bit cache gives f16 or bf16 outputs (its weights are rounded to f16)");
  DeviceGuard g(t->device);
  if (!g.ok) return fail(DEC_ECUDA, "the plan's device cannot be made current");
  TreeAttendArgs a{};
  a.m = t->meta;
  a.d = pool_dims(t);
  a.q = q;
  a.ldq = ldq;
  a.ldo = ldo;
  a.out = out;
  a.q_type = q_type;
  a.out_type = out_type;
  a.layer = layer;
  a.kv = t->slabs;
  a.scales = t->scales;
  a.part = (float*)(t->ws + t->lay.part);
  a.scale_log2 = (float)(1.4426950408889634074 / std::sqrt((double)c.head_dim));
  cudaStream_t st = (cudaStream_t)stream;
  TREE_CUDA(t->kernel == kTreeFfma  ? launch_tree_attend_f32(a, t->ctas, st)
            : t->kernel == kTreeMmaQ8 ? launch_tree_attend_q8(a, t->kv_type, &t->tm, t->ctas, st)
            : t->kernel == kTreeMma ? launch_tree_attend_f16(a, &t->tm, t->ctas, st)
                                    : launch_tree_attend_tc(a, t->kv_type, t->q8 ? &t->tm : &t->tm_groups, t->ctas, t->kernel == kTreeTcWide, st));
  // nothing to join: no second launch, unless a replay may meet a plan that has something
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (t->n_merges == 0) TREE_CUDA(cudaStreamIsCapturing(st, &cap));
  if (t->n_merges > 0 || cap != cudaStreamCaptureStatusNone) TREE_CUDA(launch_tree_merge(a, t->n_merges, t->max_parts, st));
  return DEC_OK;
}

int dec_tree_commit(dec_tree* t, const int32_t* draft, const int32_t* target, const int32_t* prior, int32_t* accepted,
                    int32_t* path, int32_t* next, void* stream) {
  int rc = check_ready(t, 0);
  if (rc) return rc;
  if (!draft || !target || !accepted || !path || !next) return fail(DEC_EINVAL, "NULL argument");
  DeviceGuard g(t->device);
  if (!g.ok) return fail(DEC_ECUDA, "the plan's device cannot be made current");
  TreeCommitArgs a{};
  a.m = t->meta;
  a.d = pool_dims(t);
  a.draft = draft;
  a.target = target;
  a.prior = prior;
  a.accepted = accepted;
  a.path = path;
  a.next = next;
  a.kv = t->slabs;
  a.kv_type = t->kv_type;
  a.scales = t->scales;
  TREE_CUDA(t->q8 ? launch_tree_commit_q8(a, (cudaStream_t)stream) : launch_tree_commit(a, (cudaStream_t)stream));
  return DEC_OK;
}

int dec_tree_read_rows(const dec_tree* t, int32_t part, int64_t* rows) {
  int rc = check_ready(t, 0);
  if (rc) return rc;
  if (!rows) return fail(DEC_EINVAL, "NULL argument");
  if (part != DEC_READ_ALL && part != DEC_READ_PAGES) return fail(DEC_EINVAL, "unknown part %d", part);
  if (t->read_rows[part] > INT32_MAX)
    return fail(DEC_ERANGE, "%lld rows are more than one call reads: read fewer sequences", (long long)t->read_rows[part]);
  *rows = t->read_rows[part];
  return DEC_OK;
}

int dec_tree_read(dec_tree* t, int32_t layer, int32_t n_layers, int32_t part, int64_t rows, int32_t out_type, void* k,
                  void* v, int64_t ld, int64_t layer_stride, void* stream) {
  int64_t have = 0;
  int rc = check_ready(t, layer);
  if (rc || (rc = dec_tree_read_rows(t, part, &have))) return rc;
  const dec_config& c = t->cfg;
  if (n_layers < 1 || n_layers > c.n_layers - layer) return fail(DEC_EINVAL, "%d layers from layer %d on are not all of the model", n_layers, layer);
  if (rows != have) return fail(DEC_EINVAL, "%lld rows asked for, the plan has %lld", (long long)rows, (long long)have);
  if (!k && !v) return fail(DEC_EINVAL, "neither keys nor values");
  for (const void* p : {k, v}) {
    if (p && (rc = check_rows(p, ld, c.n_kv_heads, c.head_dim, out_type, p == k ? "k" : "v"))) return rc;
  }
  if (k == v) return fail(DEC_EINVAL, "keys and values must not overlap");
  // layers must not run into each other; one alone has no stride
  if (n_layers > 1 && (layer_stride % 4 || layer_stride < (rows - 1) * ld + (int64_t)c.n_kv_heads * c.head_dim))
    return fail(DEC_EINVAL, "layers of %lld rows overlap at a stride of %lld, or it is no multiple of 4", (long long)rows, (long long)layer_stride);
  DeviceGuard g(t->device);
  if (!g.ok) return fail(DEC_ECUDA, "the plan's device cannot be made current");
  TreeReadArgs a{};
  a.m = t->meta;
  a.d = pool_dims(t);
  a.kv = t->slabs;
  a.scales = t->scales;
  a.kv_type = t->kv_type;
  a.out_type = out_type;
  a.layer = layer;
  a.n_layers = n_layers;
  a.part = part;
  a.rows = rows;
  a.ld = ld;
  a.layer_stride = n_layers > 1 ? layer_stride : 0;
  a.k = k;
  a.v = v;
  a.n_blocks = t->read_blocks[part];
  TREE_CUDA(launch_tree_read(a, (cudaStream_t)stream));
  return DEC_OK;
}

}  // extern "C"
