// tree.h - draft trees over the paged KV cache: what the host plan (tree.cu)
// uploads, and the launchers of the tree kernels (internal to libdec).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "optin.h"

namespace dec {

constexpr int kTreeMaxNodes = 256;  // nodes per sequence (a row of the ancestor mask is at most 8 words)
constexpr uint32_t kErrShape = 16u; // a captured call met a plan of another shape (mirrors DEC_DEV_SHAPE)

constexpr uint32_t kErrNonFinite = 32u;  // a value that is not finite was quantised (mirrors DEC_DEV_NONFINITE)

// Element types of the callers' tensors and of the cache (mirror DEC_T_*).
enum TreeType { kTreeF32 = 0, kTreeF16 = 1, kTreeBf16 = 2, kTreeE4m3 = 3, kTreeI8 = 4 };

// Header words of the uploaded plan.
enum TreeHdr { kHdrSeqs = 0, kHdrTokens, kHdrWords, kHdrRowTile, kHdrMerges, kHdrPages, kHdrRows, kHdrInts = 16 };  // two row counts

// A sequence with nodes, as the attention kernels read it (one 16-byte load).
struct alignas(16) TreeSeq {
  int32_t node0, nodes, ctx, tab;  // first node, nodes, cached tokens, first entry in tables
};
// Attention work of one CTA: `count` key tiles in the order (entry of seqs, KV
// head, row tile, key tile), from `tile` of this unit on.  A row tile is
// followed by row_tile + step of the same head while there is one, then by the
// next head's row_tile % step.
struct alignas(16) TreeCut {
  int32_t q, head, row_tile, tile;
  int32_t count, step;
  int32_t follow;  // CTAs cta + step, cta + 2 step, .. that finish this one's last unit, for this one to join
  int32_t awaited; // its first unit's part is joined by the CTA that starts that unit
  TreeSeq s;  // seqs[q]: a CTA starts with a single read
};
// A unit (sequence, KV head, row tile) that CTAs c0, c0 + stride, .., c1 share.
struct alignas(16) TreeMerge {
  int32_t head, row_tile, c0, c1;
  int32_t stride, node0, nodes, pad;
};
// A block that nodes lie in: `nodes` of them from node0 on in its slots from slot0 on (slots in front of slot0: cached tokens).
struct alignas(16) TreePage {
  int32_t block, node0, slot0, nodes;
};
// What dec_tree_read goes by, for every sequence: its tables, slots, and by part (all slots; from the first node's block on)
// the blocks and rows of the sequences before it (the entry behind the last has the sums).
struct alignas(16) TreeReadSeq {
  int32_t tab, ctx, nodes, pad;
  int32_t blocks[2], rows[2];
};

// The plan on the device: one upload, arrays back to back.
struct TreeMeta {
  const int32_t* hdr;        // [kHdrInts]
  const int32_t* seq_start;  // [S+1]
  const TreeSeq* seqs;       // the sequences with nodes, in the order of the attention work
  const int32_t* pos;        // [N] rotary position; -1: a padding node
  const int32_t* dst;        // [N] pool block * 16 + slot
  const int32_t* parents;    // [N] parent within the sequence, -1 root, -2 padding
  const uint32_t* anc;       // [N, words] bit j: the node sees node j (itself included)
  const TreeCut* cuts;       // [CTAs]
  const TreeMerge* merges;   // [hdr[kHdrMerges]]
  const TreePage* pages;     // [hdr[kHdrPages]] (8-bit caches)
  const TreeReadSeq* reads;  // [S+1]
  const int32_t* tables;     // pool block ids, sequence after sequence
  uint32_t* err;             // device error word
  uint32_t* flags;           // a word per place, 1: its part of a shared unit is there; 0 between calls
  int S, N, words, row_tile; // the shape the launch was made for (checked against hdr)
  int tile_keys;             // keys per attention tile
};

struct TreePoolDims {
  int H, Hkv, D, n_layers, n_blocks;
  int gs;  // query heads per KV head: 1 << gs (a config has 1, 2 or 4)
  float eps;
};

struct TreeAppendArgs {
  TreeMeta m;
  TreePoolDims d;
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv, ldo;
  const float *q_norm, *k_norm;
  const float* rope;  // [positions, rot/2, 2] (cos, sin); null: no rotation
  int rot, interleaved, rope_positions;
  void* q_out;
  int in_type, q_type, kv_type, layer;
  void* kv;
  float* scales;  // of an 8-bit cache: [layers][blocks][Hkv][2]
  int n_pages;    // of the plan that is set (a replay may meet another number)
  int sms;  // of the plan's device
};
cudaError_t launch_tree_append(const TreeAppendArgs& a, cudaStream_t s);
cudaError_t launch_tree_append_q8(const TreeAppendArgs& a, cudaStream_t s);

struct TreeAttendArgs {
  TreeMeta m;
  TreePoolDims d;
  const void* q;
  int64_t ldq, ldo;
  void* out;
  int q_type, out_type, layer;
  const void* kv;
  const float* scales;  // of an 8-bit cache
  float* part;  // [CTAs, 2, row_tile, D + 2] records
  float scale_log2;  // log2(e) / sqrt(D)
};
// The attention kernel for sequences of up to max_rows (nodes x query heads
// per KV head) rows, and its tiles.
enum TreeKernel { kTreeFfma = 0, kTreeMma, kTreeTc, kTreeTcWide, kTreeMmaQ8 };
struct TreeVariant {
  int kernel, row_tile, tile_keys, ctas_per_sm;
  int unit_cost;  // what starting and finishing a unit costs a CTA, in key tiles
  int join;       // shared units per hundred CTAs from which on joining in place beats a second kernel; 0: never
  int spare;      // places of the last full round that no CTA is launched for
};
constexpr int kTreeMaxCtasPerSm = 3;
cudaError_t launch_tree_attend_f32(const TreeAttendArgs& a, int ctas, cudaStream_t s);
cudaError_t launch_tree_attend_f16(const TreeAttendArgs& a, const CUtensorMap* tm, int ctas, cudaStream_t s);
cudaError_t launch_tree_attend_tc(const TreeAttendArgs& a, int kv_type, const CUtensorMap* tm, int ctas, bool wide, cudaStream_t s);
cudaError_t launch_tree_attend_q8(const TreeAttendArgs& a, int kv_type, const CUtensorMap* tm, int ctas, cudaStream_t s);
cudaError_t launch_tree_merge(const TreeAttendArgs& a, int n_merges, int parts, cudaStream_t s);

struct TreeCommitArgs {
  TreeMeta m;
  TreePoolDims d;
  const int32_t *draft, *target, *prior;
  int32_t *accepted, *path, *next;
  void* kv;
  int kv_type;
  float* scales;
};
cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t s);
cudaError_t launch_tree_commit_q8(const TreeCommitArgs& a, cudaStream_t s);

struct TreeReadArgs {
  TreeMeta m;
  TreePoolDims d;
  const void* kv;
  const float* scales;
  int kv_type, out_type, layer, n_layers, part;
  int64_t rows, ld, layer_stride;
  void *k, *v;
  int n_blocks;  // of the sequences, of the plan that is set
};
cudaError_t launch_tree_read(const TreeReadArgs& a, cudaStream_t s);

cudaError_t launch_tree_join_test(const TreeMeta& m, int late, uint64_t limit_ns, cudaStream_t s);

constexpr int kRopeMaxPairs = 64;
struct RopeTableArgs {
  float* table;
  int positions, pairs;
  double mult;
  double freq[kRopeMaxPairs];
};
cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t s);

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while its predecessor drains and waits for it before its first access.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*k)(P...), int grid, int block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace dec
