// hw_decode_plan.cuh - what the tensor-core decode kernels (attn_decode_tc.cu,
// attn_decode_fp4.cu) share: the plan of a step as hw_attn_plan leaves it in the workspace,
// the walk over a CTA's units, the query-side metadata of a segment.
#pragma once

#include <cuda_bf16.h>

#include "hw_device.cuh"
#include "hw_sm100.cuh"

namespace hw {

using namespace sm100;

namespace {

constexpr int kStages = 3;  // first tiles of a CTA that a plan decodes (bf16: the ring's stages)
constexpr int kT = kTcTile;                   // 128 tokens per tile
constexpr int kN = kMaxQ;                     // 32 query heads per tile (MMA N)
constexpr int kPre = 4;  // slots of query-side segment metadata
constexpr int kPreList = 64;  // records of a merge list built ahead of the merge
constexpr int kPreItems = 2;  // merge items of a CTA whose lists a plan builds
constexpr int kAppList = 8;   // new tokens of a CTA a plan lists (more: found by a scan)

// Query-side metadata of a segment: its view references and q heads, and per
// query column qi = (reference qi / G, q head qi % G) the q row to read and
// the rotation i_q - offset of its reference.
struct SegQ {
  SegMeta m;
  int32_t qrow[kMaxQ];  // row * Hq + q head
  int32_t minlim;       // fewest tokens of the block a column attends (view limits), <= len
  int64_t rel[kMaxQ];
};

// What the plan derives for one CTA (copied as one block).
struct alignas(16) CtaPlan {
  int64_t u0, u1;          // its units
  int64_t us[kPre];        // first unit of its segments 0 .. kPre-1 (u1 where none)
  SegQ pre[kPre];          // query-side metadata of segment j in pre[j % kPre]
  int32_t mpre[kPreItems][kPreList];  // record lists of its first merge items
  int32_t mpre_n[kPreItems];          // their lengths, or -1 (not built)
  int32_t mrank;           // its rank among the CTAs by units (merge_ctas: it merges if < nm)
  int32_t c_log;           // the split's CTA index of this work (see "plans": the order of
                           // the records is by rank, so a launch's CTA b runs rank b)
  int32_t trow[kStages];   // its first tiles (the ring's first fill): first cache row,
  uint8_t th[kStages];     // kv head,
  uint8_t tfl[kStages];    // segment flags (see TileRef)
  uint8_t n_first;         // how many (min(kStages, u1 - u0)); 0 without a plan
  int32_t app_n;           // new tokens this CTA writes (hw_attn_plan_append), 0: none
  int32_t app_tile;        // its first tile (from u0) that holds one of them
  // the first kAppList of them: (row * Hkv + kv head), cache row, block-local position
  int32_t app_pair[kAppList], app_row[kAppList], app_pos[kAppList];
};

// ------------------------------------------------------------------- plans
//
// hw_attn_plan runs plan_kernel once per decode step: it copies the metadata
// into the workspace and, for this kernel, writes what every launch of the
// step would otherwise derive again - a header, the shared plan (PlanShared:
// unit prefix and metadata cache with ranks) and one CtaPlan per CTA (unit
// range, first segments' query metadata, first merge list).  A planned
// launch copies the shared part and its own record into shared memory with
// two bulk copies and starts streaming at once.

constexpr uint32_t kPlanMagic = 0x4c505748u;  // "HWPL"

struct PlanHeader {
  uint32_t magic;
  int32_t grid, n_rows, n_q_heads, n_kv_heads, head_dim, n_blocks, n_view;
  int64_t capacity;
  int32_t limited;  // planned with view limits: decoded by the limited kernel only
};
static_assert(sizeof(PlanHeader) <= kPlanHeaderBytes, "plan header");
static_assert(sizeof(PlanShared) % 16 == 0 && sizeof(CtaPlan) % 16 == 0, "bulk copy sizes");

__device__ __forceinline__ const uint8_t *plan_cta_record(const uint8_t *plan, int c) {
  return plan + kPlanHeaderBytes + sizeof(PlanShared) + static_cast<size_t>(c) * sizeof(CtaPlan);
}

// The launch's RoPE table (MetaCache::phase, the first field of the shared
// part's metadata) is written into shared memory at the kernel's entry: the
// plan copies skip those bytes.
constexpr uint32_t kPhaseOff = offsetof(PlanShared, cache) + offsetof(MetaCache, phase);
constexpr uint32_t kPhaseBytes = sizeof(MetaCache::phase);
static_assert(kPhaseOff % 16 == 0 && kPhaseBytes % 16 == 0, "the phase table is a whole number of 16-B chunks");

// Does a plan header describe a launch of `grid` CTAs with these arguments?
__device__ __forceinline__ bool header_matches(const DecodeArgs &a, const PlanHeader &h, int grid) {
  return h.magic == kPlanMagic && h.grid == grid && h.n_rows == a.n_rows &&
         h.n_q_heads == a.n_q_heads && h.n_kv_heads == a.n_kv_heads && h.head_dim == a.head_dim &&
         h.n_blocks == a.n_blocks && h.n_view == a.n_view && h.capacity == a.capacity &&
         (h.limited != 0) == (a.view_limit != nullptr);
}


__device__ __forceinline__ bool seg_first_unit(const UnitPos &x, int64_t u, int64_t u0) {
  return u == u0 || u == x.seg_first;
}
__device__ __forceinline__ bool seg_last_unit(const UnitPos &x, int64_t u, int64_t u1) {
  return u + 1 == u1 || u + 1 == x.seg_first + x.tiles;
}

// The tile of unit u in a CTA's range [u0, u1): its first cache row, its kv
// head, and whether it starts (1) / ends (2) its segment within the range.
struct TileRef {
  int row, h;
  uint8_t flags;
};
__device__ __forceinline__ TileRef tile_ref(const PlanCore &P, int n_blocks, int64_t u, int64_t u0,
                                            int64_t u1) {
  const UnitPos x = unit_pos(P, n_blocks, u);
  TileRef t;
  t.row = P.start[x.b] + x.t * kT;
  t.h = x.h;
  t.flags = (seg_first_unit(x, u, u0) ? 1 : 0) | (seg_last_unit(x, u, u1) ? 2 : 0);
  return t;
}

// The tokens of its block that view entry e attends: all len, or fewer under
// a view limit.
__device__ __forceinline__ int entry_limit(const int32_t *view_limit, int e, int len) {
  if (!view_limit) return len;
  const int v = __ldg(view_limit + e);
  return v >= 0 && v < len ? v : len;
}

// Query-side metadata of segment (block b, column group g, kv head h) into X, by one warp (shared memory
// only, except for views beyond the metadata cache), with the fewest tokens
// any of its columns attends (len when no view limit cuts the block).
template <bool kLimit>
__device__ void seg_pre(const DecodeArgs &a, const PlanCore &P, const MetaCache &C, SegQ &X, int b,
                        int g, int h, int lane) {
  const int len = P.len[b];
  const int G = a.n_q_heads / a.n_kv_heads;
  gather_refs(a, C, X.m, b, g, lane);
  gather_qheads(a, C, X.m, h, lane);
  __syncwarp();
  int lim = len;
  if (lane < X.m.n_ref * G) {
    const int e = X.m.ref_entry[lane / G];
    X.qrow[lane] = (e / a.n_view) * a.n_q_heads + X.m.qhead[lane % G];
    X.rel[lane] = entry_rel(a, C, e);
    if (kLimit) lim = entry_limit(a.view_limit, e, len);
  }
  if (kLimit) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) lim = min(lim, __shfl_xor_sync(0xffffffffu, lim, o));
  }
  if (lane == 0) X.minlim = lim;
  __syncwarp();
}

// One item of the rotated queries: column qi, elements 8c..8c+7 and their
// RoPE partners 64+8c..64+8c+7, and the column's rotation i_q - offset.  Only
// columns below nq are rotated: the rows of Q~ past them feed S columns that
// the softmax neither reads nor lets into P (their P is zero).
struct QItem {
  uint4 lo, hi;
  int64_t rel;
};
__device__ __forceinline__ void load_item(const DecodeArgs &a, const SegQ &X, int qi, int c,
                                          QItem &it) {
  const __nv_bfloat16 *qp = reinterpret_cast<const __nv_bfloat16 *>(a.q) +
                            static_cast<int64_t>(X.qrow[qi]) * 128;
  it.lo = __ldg(reinterpret_cast<const uint4 *>(qp + 8 * c));
  it.hi = __ldg(reinterpret_cast<const uint4 *>(qp + 64 + 8 * c));
  it.rel = X.rel[qi];
}

// First unit after the segment that holds unit u.
__device__ __forceinline__ int64_t next_segment(const PlanCore &P, int n_blocks, int64_t u) {
  const UnitPos x = unit_pos(P, n_blocks, u);
  return x.seg_first + x.tiles;
}

// Max over a warp of a non-negative float.
__device__ __forceinline__ float warp_max_nonneg(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}


}  // namespace

}  // namespace hw
