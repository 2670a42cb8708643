// hw_tree.h - the draft-tree operators' plan: its layout in a workspace, and
// the arguments their kernels share.  Not part of the public interface.
//
// A step's plan is built once by launch_tree_plan (tree_plan.cu) and read by
// every layer's launches:
//   column   = one query of a kv head: a row's node and one of the kv head's q
//              heads.  Columns are numbered row by row, node by node.
//   group    = up to `cols` neighbouring columns, attended together: every K/V
//              tile that one of them sees is read once for all of them.
//              Neighbouring rows join one group as long as they share a block.
//   span     = the tokens of a block that rows of the group see, or of one
//              row's tree.  A group's blocks come by number (a block that a
//              row names twice, twice), then its rows' trees.  From span to
//              span only the queries' rotation changes; the softmax goes on.
//   unit     = one tile of `tile` tokens of a span for one kv head; units are
//              ordered by kv head, group, span and tile, on a weighted line,
//              first those of the groups with over 128 columns, which need a
//              CTA's shared memory laid out otherwise (n_wide groups; they come
//              first by number as well), then the others'; no CTA has both:
//              a tile weighs tile1 or tile2 (over 128 columns), the first tile
//              of a span `span` more (a tree's `tree` more still), that of a
//              group `group` more.  CTA
//              c of C takes the units that start in [c W / C, (c + 1) W / C) of
//              its kind's part; shares without a unit get no CTA.
//   record   = what a CTA leaves for (kv head, group): per column the running
//              maximum m and sum l of the softmax (log2 domain) and the
//              unnormalised output.  The records of one (kv head, group) lie
//              behind one another, CTA after CTA.  Within a record 8 output
//              elements (32 bytes, a sector) of every column lie side by
//              side, then the next 8: a thread that owns a column and a warp
//              that owns a row both move whole sectors.
// The rotation of a (row, view entry, node) is the same for every layer and q
// head: the plan holds its cos and sin, head_dim / 2 pairs each - in fp32 for
// the keys that are stored and for the CUDA cores, and again in the order
// in which the tensor-core kernel reads them (turn_at): in fp32 for bf16 caches,
// whose turned queries keep 16 bits, in fp16 for E4M3 caches, whose keep 8.
// tree_merge_kernel joins the records of every (row, node, q head).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hogwild.h"

namespace hw {

constexpr uint32_t kTreeMagic = 0x48577472u;
constexpr int kMaxNodes = HW_MAX_TREE_NODES;
// The running maximum before any score: finite, so that what sees nothing gets
// weights of 0, and what sees only NaN a sum of NaN, not none.
constexpr float kNoScore = -3.402823466e38f;

struct TreeHeader {
  uint32_t magic;
  int32_t n_rows, max_nodes, n_q_heads, n_kv_heads, head_dim, n_blocks, n_view, dtype;
  int32_t n_groups;  // per kv head
  int32_t n_ctas;    // CTAs with units (0: nothing to attend)
  int32_t streams;   // records that a CTA leaves of a group with up to 128 columns
  int32_t n_col_blocks;  // entries of the merge's table: (group, first column) of 32 columns
  int32_t n_wide;        // groups with over 128 columns (per kv head; the first ones)
  int64_t capacity;
  double rope_theta;  // of the rotations that the plan holds
};

struct TreeGroup {
  int32_t row0, row1;      // first and last row with columns in the group
  int32_t rank0, n_rows;   // rows with nodes before row0; such rows in the group
  int32_t col0, n_cols;    // its columns (numbered over all rows)
  int32_t span0, n_spans;
};
struct TreeSpan {
  int32_t start, len;  // pool tokens
  int32_t row;         // the row whose tree this is, or -1: a block
  int32_t map;         // block: in the map, per row of the group its view entry, or -1
  int32_t tile0;       // tiles of the group before it
  int32_t partial;     // not every column sees every token of it
};
struct TreeColumn {
  int32_t node, head;   // row * max_nodes + node; q head within its kv head's
  int32_t rot;          // table row of the rotation for view entry 0; entry v's lies v * n_nodes further
  uint16_t n_nodes, row;  // of its row; the row's number among the group's rows
};
struct TreeCta {
  int32_t head, group, span, tile, n_units;  // first unit and count
  int32_t wide;                              // its groups have over 128 columns (all or none)
  TreeGroup g;                               // copies: one load instead of three in a row
  TreeSpan sp;
};

// Byte offsets of the plan's arrays in the workspace (the error word is at 0).
struct TreeLayout {
  size_t hdr, groups, wbase, spans, map, columns, rot, turns, blocks, piece_row, piece_cta, ctas;
  size_t n_nodes, slot, pos, end, col, rot0, rank, depth, mask, heads, block_start, block_len;
  size_t ml, o, total;
  int64_t max_groups, max_spans, max_map, max_cols, max_blocks, max_rots, max_rows;
  int32_t cols, tile, ctas_max;
};

struct TreeArgs {
  const void *q, *k_new, *v_new;
  void *k, *v;
  const float *k_scale, *v_scale;
  void *out;
  float *lse;
  uint8_t *ws;
  TreeLayout L;
  int32_t n_rows, max_nodes, n_q_heads, n_kv_heads, head_dim, n_blocks, n_view, dtype;
  int64_t capacity;
  double rope_theta;
  float scale_log2;
  uint64_t phase[64];  // RoPE phase table (hw_internal.h)
};

// The caller's metadata of a step (device pointers).
struct TreeMeta {
  const int32_t *block_start, *block_len, *view_block, *view_offset, *q_pos, *q_to_kv;
  const int32_t *tree_block, *tree_start, *n_nodes, *parent;
};

struct TreeCommitArgs {
  void *k, *v;
  const int32_t *path, *n_path;
  int32_t n_layers, elem_bytes;
};

struct TreeVerifyArgs {
  const void *p, *q;
  int64_t p_stride, q_stride;
  const int32_t *n_nodes, *parent, *token;
  const float *u_accept, *u_sample;
  int32_t *path, *n_path, *next_token;
  int32_t n_rows, max_nodes, vocab, dtype;
  int32_t keep;  // slices fit shared memory (set by the launch)
};

TreeLayout tree_layout(const hw_attn_desc &d, int max_nodes, int sms);
// Whether these caches run on the tensor cores.
inline bool tree_on_tensor_cores(int dtype, int head_dim) {
  return (dtype == HW_BF16 || dtype == HW_FP8_E4M3) && head_dim == 128;
}

cudaError_t launch_tree_plan(const TreeArgs &a, const TreeMeta &m, cudaStream_t s);
cudaError_t launch_tree_append(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_tc(const TreeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s);
cudaError_t launch_tree_merge(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_commit(const TreeArgs &a, const TreeCommitArgs &c, cudaStream_t s);
cudaError_t launch_tree_verify(const TreeVerifyArgs &a, cudaStream_t s);

#ifdef __CUDACC__
// Where a table row keeps element e's (cos, sin), e < half = head_dim / 2:
// the n that 16 bytes hold (4 in fp16, 2 in fp32) side by side, 8c + n j ..
// 8c + n j + n - 1, c running before j, so that the lanes that each turn 8
// neighbouring elements read neighbouring memory.
__host__ __device__ __forceinline__ int turn_at(int e, int half, int n) {
  return ((e & 7) / n * (half >> 3) + (e >> 3)) * n + e % n;
}
// Element d of column col in a record of n_cols columns that starts at row rec.
__device__ __forceinline__ int64_t record_at(int64_t rec, int n_cols, int col, int d, int D) {
  return rec * D + static_cast<int64_t>(d >> 3) * n_cols * 8 + col * 8 + (d & 7);
}
template <typename T>
__device__ __forceinline__ T *tree_at(const TreeArgs &a, size_t off) {
  return reinterpret_cast<T *>(a.ws + off);
}
// The group behind one on the unit line; head may come to n_kv_heads behind the last.
__device__ __forceinline__ void next_group(const TreeHeader &h, int &head, int &group) {
  if (++group == h.n_wide) {
    group = 0;
    if (++head == h.n_kv_heads && h.n_wide < h.n_groups) head = 0, group = h.n_wide;
  } else if (group == h.n_groups) {
    group = h.n_wide;
    ++head;
  }
}
// The plan in the workspace is one of this description.
__device__ __forceinline__ bool tree_plan_ok(const TreeArgs &a) {
  const TreeHeader &h = *tree_at<const TreeHeader>(a, a.L.hdr);
  return h.magic == kTreeMagic && h.n_rows == a.n_rows && h.max_nodes == a.max_nodes &&
         h.n_q_heads == a.n_q_heads && h.n_kv_heads == a.n_kv_heads && h.head_dim == a.head_dim &&
         h.n_blocks == a.n_blocks && h.n_view == a.n_view && h.dtype == a.dtype &&
         h.capacity == a.capacity && h.rope_theta == a.rope_theta;
}
#endif

}  // namespace hw
