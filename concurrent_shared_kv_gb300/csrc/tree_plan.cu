// tree_plan.cu - the draft-tree operators' plan (hw_tree.h), the write of the
// drafted tokens into the cache, the merge of the partial results, and the
// commit of an accepted path.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "hw_device.cuh"
#include "hw_tree.h"

namespace hw {

namespace {

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Weights of the unit line, measured on the tensor-core kernel (a fit of its
// CTAs' times, then tried out) in steps of about 420 clocks: a tile against up
// to 128 columns and against more, what a span's new queries and empty pipeline
// cost beside its tiles, a tree's more of that, a group's records.  (For bf16
// tile2 7, 8, 9: 4 trees of 16 nodes over 16K 47.1, 45.6, 43.2 us; group 22 and
// 16: a ragged batch, over five seeds, 160 and 156 us.)  On the CUDA cores tiles
// outweigh the rest.  Where every unit can have a CTA of its own, each does:
// the units then weigh the same.
struct TreeCost {
  int32_t tile1, tile2, span, tree, group;
};
__device__ inline TreeCost tree_cost(int cols, bool e4m3, bool alone) {
  if (alone) return TreeCost{1, 1, 0, 0, 0};
  if (cols <= 128) return TreeCost{4, 4, 1, 0, 1};
  return e4m3 ? TreeCost{6, 12, 27, 0, 8} : TreeCost{4, 9, 17, 8, 16};
}

struct TreePlanSmem {
  int32_t len[HW_MAX_BLOCKS], start[HW_MAX_BLOCKS];
  int64_t scan[kPlanWarps + 1];
  int64_t carry;
  int64_t uidx[1025];
  int16_t number[kPlanThreads];  // of every share with units
  int32_t ok, n_groups, n_wide, n_spans, n_map;
  union {
    uint8_t parent[kPlanWarps][kMaxNodes];
    uint8_t count[kPlanWarps][HW_MAX_BLOCKS];  // of a group: the most often a row names the block
  };
  int16_t first[kPlanWarps][HW_MAX_BLOCKS];    // of a group: the block's first span
  int16_t vb[HW_MAX_VIEW_ENTRIES];    // block of every view entry with tokens, -1: none
  uint8_t nodes[HW_MAX_VIEW_ENTRIES];  // nodes of every row (rows <= HW_MAX_VIEW_ENTRIES)
  uint8_t apart[HW_MAX_VIEW_ENTRIES];  // the row shares no block with the one before it
};

// Exclusive prefix sum over the CTA; returns this thread's prefix and adds
// the total to S.carry (read by every thread before the next call).
__device__ int64_t block_scan(TreePlanSmem &S, int64_t x) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) S.scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int64_t w = S.scan[lane];
    int64_t wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += y;
    }
    S.scan[lane] = wi - w;
    if (lane == 31) S.scan[kPlanWarps] = wi;
  }
  __syncthreads();
  const int64_t r = S.carry + S.scan[warp] + incl - x;
  __syncthreads();
  if (threadIdx.x == 0) S.carry += S.scan[kPlanWarps];
  __syncthreads();
  return r;
}

// A row's tree as the caller gives it: its first pool token, or -1.
__device__ __forceinline__ int64_t tree_slot(const TreeMeta &m, int n_blocks, int r) {
  if (m.tree_start) return m.tree_start[r];
  const int b = m.tree_block[r];
  if (b < 0 || b >= n_blocks) return -1;
  return static_cast<int64_t>(m.block_start[b]) + m.block_len[b];
}

__device__ __forceinline__ bool ranges_meet(int64_t a, int64_t na, int64_t b, int64_t nb) {
  return na > 0 && nb > 0 && a < b + nb && b < a + na;
}

// One row, by one warp: its checks but for the other rows' trees (tree_meets),
// depths and ancestor masks.  Returns its node count (0 if the row is refused).
__device__ int plan_row(const TreeArgs &a, const TreeMeta &m, TreePlanSmem &S, int32_t *err, int r,
                        int lane) {
  const int T = a.max_nodes;
  const int n = m.n_nodes[r];
  if (n == 0) return 0;
  if (n < 0 || n > T) {
    if (lane == 0) flag_error(err, HW_DEV_BAD_TREE);
    return 0;
  }
  const int b = m.tree_block[r];
  if (b < 0 || b >= a.n_blocks) {
    if (lane == 0) flag_error(err, HW_DEV_BAD_BLOCK);
    return 0;
  }
  // the nodes' tokens: inside the pool, outside every block
  const int64_t slot = tree_slot(m, a.n_blocks, r);
  bool bad_range = S.len[b] < 0 || slot < 0 || slot + n > a.capacity;
  for (int x = lane; x < a.n_blocks; x += 32)
    bad_range |= ranges_meet(slot, n, S.start[x], S.len[x]);
  // parents before their children
  uint8_t *par = S.parent[threadIdx.x >> 5];
  bool bad_tree = false;
  for (int i = lane; i < n; i += 32) {
    const int p = m.parent[static_cast<int64_t>(r) * T + i];
    bad_tree |= p < -1 || p >= i;
    par[i] = p < 0 ? 255 : static_cast<uint8_t>(p);
  }
  bad_tree = __any_sync(0xffffffffu, bad_tree);
  bad_range = __any_sync(0xffffffffu, bad_range);
  if (bad_tree || bad_range) {
    if (lane == 0) flag_error(err, (bad_tree ? HW_DEV_BAD_TREE : 0) | (bad_range ? HW_DEV_BAD_RANGE : 0));
    __syncwarp();
    return 0;
  }
  for (int i = lane; i < n; i += 32) {
    uint32_t w[4] = {0, 0, 0, 0};
    int d = -1;
    for (int x = i; x != 255; x = par[x]) {  // up to the root: parents have lower indices
      w[x >> 5] |= 1u << (x & 31);
      ++d;
    }
    tree_at<uint4>(a, a.L.mask)[static_cast<int64_t>(r) * T + i] = make_uint4(w[0], w[1], w[2], w[3]);
    tree_at<int32_t>(a, a.L.depth)[static_cast<int64_t>(r) * T + i] = d;
  }
  if (lane == 0) {
    tree_at<int32_t>(a, a.L.slot)[r] = static_cast<int32_t>(slot);
    tree_at<int32_t>(a, a.L.pos)[r] = S.len[b];
    tree_at<int32_t>(a, a.L.end)[r] = S.start[b] + S.len[b];
  }
  __syncwarp();
  return n;
}

// Whether the row's tree meets that of another row which takes part, as far as
// plan_row can tell.  By one warp.
__device__ bool tree_meets(const TreeArgs &a, const TreePlanSmem &S, int r, int lane) {
  const int32_t *slot = tree_at<int32_t>(a, a.L.slot);
  bool meets = false;
  if (S.nodes[r] > 0)
    for (int x = lane; x < a.n_rows; x += 32)
      if (x != r && S.nodes[x] > 0) meets |= ranges_meet(slot[r], S.nodes[r], slot[x], S.nodes[x]);
  return __any_sync(0xffffffffu, meets);
}

// The CTA that owns a unit starting at weight w.
__device__ __forceinline__ int cta_of_weight(int64_t w, int64_t W, int C) {
  return static_cast<int>(((w + 1) * C - 1) / W);
}

// How often the row names entry v's block before v, and whether v is the last.
__device__ __forceinline__ int entry_rank(const TreePlanSmem &S, int e0, int v, int V, bool *last) {
  const int b = S.vb[e0 + v];
  int k = 0;
  *last = true;
  for (int x = 0; x < V; ++x)
    if (x != v && S.vb[e0 + x] == b) {
      if (x < v) ++k; else *last = false;
    }
  return k;
}

// Rows into groups: their columns one behind another, cut where a row shares
// no block with the one before it and every a.L.cols columns.  One thread.
__device__ void plan_groups(const TreeArgs &a, TreePlanSmem &S) {
  const int R = a.n_rows, V = a.n_view, G = a.n_q_heads / a.n_kv_heads, CG = a.L.cols;
  TreeGroup *groups = tree_at<TreeGroup>(a, a.L.groups);
  int col = 0, rank = 0, rot = 0, n = 0, n_wide = 0;
  TreeGroup g = {};
  g.n_cols = CG;
  const auto done = [&] {
    if (n == 0) return;
    groups[n - 1] = g;
    n_wide += g.n_cols > 128;
  };
  for (int r = 0; r < R; ++r) {
    const int nodes = S.nodes[r];
    tree_at<int32_t>(a, a.L.col)[r] = col;
    tree_at<int32_t>(a, a.L.rank)[r] = rank;
    tree_at<int32_t>(a, a.L.rot0)[r] = rot;
    if (nodes == 0) continue;
    if (S.apart[r]) {
      done();
      g.n_cols = CG;
    }
    for (int left = nodes * G; left > 0;) {
      if (g.n_cols == CG) {
        if (!(S.apart[r] && left == nodes * G)) done();
        g = TreeGroup{r, r, rank, 0, col, 0, 0, 0};
        ++n;
      }
      const int take = min(left, CG - g.n_cols);
      g.n_cols += take;
      g.row1 = r;
      g.n_rows = rank + 1 - g.rank0;
      col += take;
      left -= take;
    }
    ++rank;
    rot += nodes * (V + 1);
  }
  done();
  S.n_groups = n;
  S.n_wide = n_wide;
}

// The n_wide groups with over 128 columns ahead of the others, each in order.
// By all threads (S.carry is 0 before and after).
__device__ void wide_first(const TreeArgs &a, TreePlanSmem &S, int n, int n_wide) {
  if (n_wide == 0 || n_wide == n) return;
  TreeGroup *groups = tree_at<TreeGroup>(a, a.L.groups);
  TreeGroup *sorted = tree_at<TreeGroup>(a, a.L.o);  // (room for records, which this step has none of yet)
  for (int g0 = 0; g0 < n; g0 += kPlanThreads) {
    const int g = g0 + threadIdx.x;
    const TreeGroup own = g < n ? groups[g] : TreeGroup{};
    const int at = static_cast<int>(block_scan(S, own.n_cols > 128));
    if (g < n) sorted[own.n_cols > 128 ? at : n_wide + g - at] = own;
  }
  if (threadIdx.x == 0) S.carry = 0;
  __syncthreads();
  for (int g = threadIdx.x; g < n; g += kPlanThreads) groups[g] = sorted[g];
  __syncthreads();
}

// A group's spans, by one warp; its number of tiles goes to ubase.
__device__ void plan_spans(const TreeArgs &a, TreePlanSmem &S, int gi, int64_t *ubase, int lane) {
  const int V = a.n_view, TL = a.L.tile, warp = threadIdx.x >> 5;
  TreeGroup &g = tree_at<TreeGroup>(a, a.L.groups)[gi];
  uint8_t *count = S.count[warp];
  int16_t *first = S.first[warp];
  for (int b = lane; b < a.n_blocks; b += 32) count[b] = 0;
  __syncwarp();
  for (int r = g.row0; r <= g.row1; ++r) {
    if (S.nodes[r] == 0) continue;
    for (int v = lane; v < V; v += 32) {
      const int b = S.vb[r * V + v];
      bool last;
      const int k = b < 0 ? 0 : entry_rank(S, r * V, v, V, &last);
      if (b >= 0 && last && k + 1 > count[b]) count[b] = static_cast<uint8_t>(k + 1);
    }
    __syncwarp();
  }
  int nb = 0;
  for (int b0 = 0; b0 < a.n_blocks; b0 += 32) {
    const int b = b0 + lane, c = b < a.n_blocks ? count[b] : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (b < a.n_blocks) first[b] = static_cast<int16_t>(nb + incl - c);
    nb += __shfl_sync(0xffffffffu, incl, 31);
  }
  const int n = nb + g.n_rows;
  int span0 = 0, map0 = 0;
  if (lane == 0) {
    span0 = atomicAdd(&S.n_spans, n);
    map0 = atomicAdd(&S.n_map, nb * g.n_rows);
    g.span0 = span0;
    g.n_spans = n;
  }
  span0 = __shfl_sync(0xffffffffu, span0, 0);
  map0 = __shfl_sync(0xffffffffu, map0, 0);
  TreeSpan *spans = tree_at<TreeSpan>(a, a.L.spans) + span0;
  int16_t *map = tree_at<int16_t>(a, a.L.map) + map0;
  for (int x = lane; x < nb * g.n_rows; x += 32) map[x] = -1;
  for (int b = lane; b < a.n_blocks; b += 32)
    for (int k = 0; k < count[b]; ++k)
      spans[first[b] + k] = TreeSpan{S.start[b], S.len[b], -1, map0 + (first[b] + k) * g.n_rows, 0, 0};
  __syncwarp();
  int j = 0;
  for (int r = g.row0; r <= g.row1; ++r) {
    if (S.nodes[r] == 0) continue;
    for (int v = lane; v < V; v += 32) {
      const int b = S.vb[r * V + v];
      bool last;
      if (b >= 0) map[(first[b] + entry_rank(S, r * V, v, V, &last)) * g.n_rows + j] = static_cast<int16_t>(v);
    }
    if (lane == 0) spans[nb + j] = TreeSpan{tree_at<int32_t>(a, a.L.slot)[r], S.nodes[r], r, 0, 0, 1};
    ++j;
  }
  __syncwarp();
  int tiles = 0;
  for (int s0 = 0; s0 < n; s0 += 32) {
    const int s = s0 + lane;
    const int t = s < n ? (spans[s].len + TL - 1) / TL : 0;
    int ti = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += y;
    }
    if (s < n) {
      spans[s].tile0 = tiles + ti - t;
      if (s < nb)
        for (int x = 0; x < g.n_rows; ++x) spans[s].partial |= map[s * g.n_rows + x] < 0;
    }
    tiles += __shfl_sync(0xffffffffu, ti, 31);
  }
  if (lane == 0) ubase[gi] = tiles;
}

// Weight of a group before its span s, which has tile0 tiles before it (its
// last n_rows spans are trees), and of what a span costs beside its tiles.
__device__ __forceinline__ int64_t span_weight(const TreeCost &c, const TreeGroup &g, int s, int tile0) {
  return s == 0 ? 0
                : c.group + static_cast<int64_t>(s) * c.span + static_cast<int64_t>(max(0, s - g.n_spans + g.n_rows)) * c.tree +
                      static_cast<int64_t>(tile0) * (g.n_cols > 128 ? c.tile2 : c.tile1);
}
__device__ __forceinline__ int span_cost(const TreeCost &c, const TreeGroup &g, int s) {
  return c.span + (s == 0 ? c.group : 0) + (s >= g.n_spans - g.n_rows ? c.tree : 0);
}

// The plan but for its tables, by one CTA.  (With the tables 23 to 35 us, once
// a step: trips to L2 and barriers, not work.)
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const __grid_constant__ TreeArgs a,
                                                                 const __grid_constant__ TreeMeta m) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  TreePlanSmem &S = *reinterpret_cast<TreePlanSmem *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.n_rows, V = a.n_view, E = R * V, T = a.max_nodes;
  const int G = a.n_q_heads / a.n_kv_heads, TL = a.L.tile;
  int32_t *err = reinterpret_cast<int32_t *>(a.ws);
  TreeHeader &hdr = *tree_at<TreeHeader>(a, a.L.hdr);
  if (tid == 0) {
    S.ok = 1;
    S.carry = 0;
    S.n_spans = S.n_map = 0;
    hdr.magic = 0;
  }
  // blocks: the usable length of each (-1: skipped)
  for (int b = tid; b < a.n_blocks; b += kPlanThreads) {
    const int st = m.block_start[b], ln = m.block_len[b];
    const bool bad = st < 0 || ln < 0 || static_cast<int64_t>(st) + ln > a.capacity;
    if (bad) flag_error(err, HW_DEV_BAD_RANGE);
    S.start[b] = bad ? 0 : st;
    S.len[b] = bad ? -1 : ln;
    tree_at<int32_t>(a, a.L.block_start)[b] = S.start[b];
    tree_at<int32_t>(a, a.L.block_len)[b] = S.len[b];
  }
  // the q heads of every kv head
  for (int h = warp; h < a.n_kv_heads; h += kPlanWarps) {
    int found = 0;
    for (int x0 = 0; x0 < a.n_q_heads; x0 += 32) {
      const int x = x0 + lane;
      const int g = x < a.n_q_heads ? (m.q_to_kv ? m.q_to_kv[x] : x / G) : -1;
      const unsigned hit = __ballot_sync(0xffffffffu, g == h);
      const int at = found + __popc(hit & lanemask_lt(lane));
      if (g == h && at < G) tree_at<int32_t>(a, a.L.heads)[h * G + at] = x;
      found += __popc(hit);
    }
    if (found != G && lane == 0) {
      flag_error(err, HW_DEV_BAD_HEADMAP);
      S.ok = 0;
    }
  }
  __syncthreads();
  for (int r = warp; r < R; r += kPlanWarps) {
    int n = plan_row(a, m, S, err, r, lane);
    if (!S.ok) n = 0;  // no usable head map: the plan attends and writes nothing
    if (lane == 0) S.nodes[r] = static_cast<uint8_t>(n);
  }
  for (int e = tid; e < E; e += kPlanThreads) {
    const int b = m.view_block[e];
    const bool bad = b < -1 || b >= a.n_blocks;
    if (bad) flag_error(err, HW_DEV_BAD_BLOCK);
    S.vb[e] = static_cast<int16_t>(bad || b < 0 || S.len[b] <= 0 ? -1 : b);
  }
  __syncthreads();
  // rows whose trees meet are refused together (apart[] holds which, for now)
  for (int r = warp; r < R; r += kPlanWarps) {
    const bool meets = tree_meets(a, S, r, lane);
    if (lane == 0) S.apart[r] = meets;
    if (meets && lane == 0) flag_error(err, HW_DEV_BAD_RANGE);
  }
  __syncthreads();
  for (int r = tid; r < R; r += kPlanThreads) {
    if (S.apart[r]) S.nodes[r] = 0;
    tree_at<int32_t>(a, a.L.n_nodes)[r] = S.nodes[r];
  }
  __syncthreads();
  for (int r = warp; r < R; r += kPlanWarps) {
    int before = r - 1;  // the row before it that takes part
    while (before >= 0 && S.nodes[before] == 0) --before;
    bool share = false;
    for (int v = lane; before >= 0 && v < V; v += 32)
      for (int x = 0; x < V; ++x) share |= S.vb[r * V + v] >= 0 && S.vb[r * V + v] == S.vb[before * V + x];
    share = __any_sync(0xffffffffu, share);
    if (lane == 0) S.apart[r] = !share;
  }
  __syncthreads();
  if (tid == 0) plan_groups(a, S);
  __syncthreads();
  const int n_groups = S.n_groups, n_wide = S.n_wide;
  wide_first(a, S, n_groups, n_wide);
  int64_t *wbase = tree_at<int64_t>(a, a.L.wbase), *ubase = wbase + a.L.max_groups;
  for (int g = warp; g < n_groups; g += kPlanWarps) plan_spans(a, S, g, ubase, lane);
  __syncthreads();
  const TreeGroup *groups = tree_at<TreeGroup>(a, a.L.groups);
  const TreeSpan *spans = tree_at<TreeSpan>(a, a.L.spans);
  // units, then weights before each group
  for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    const int64_t at = block_scan(S, g < n_groups ? ubase[g] : 0);
    if (g < n_groups) ubase[g] = at;
  }
  const int64_t UH = S.carry, U = UH * a.n_kv_heads;
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  const TreeCost cost = tree_cost(a.L.cols, a.dtype == HW_FP8_E4M3, U <= a.L.ctas_max);
  for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    const int64_t tiles = g < n_groups ? (g + 1 < n_groups ? ubase[g + 1] : UH) - ubase[g] : 0;
    const int64_t at = block_scan(S, g < n_groups ? span_weight(cost, groups[g], groups[g].n_spans, static_cast<int>(tiles)) : 0);
    if (g < n_groups) wbase[g] = at;
  }
  const int64_t WH = S.carry, W = WH * a.n_kv_heads;
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  // a kv head's wide groups: their weight and units
  const int64_t WW = n_wide < n_groups ? wbase[n_wide] : WH, UW = n_wide < n_groups ? ubase[n_wide] : UH;
  const auto weight_before = [&](int h, int g) {  // on the line
    return g < n_wide ? h * WW + wbase[g] : (a.n_kv_heads - 1 - h) * WW + h * WH + wbase[g];
  };
  const auto units_before = [&](int h, int g) {
    return g < n_wide ? h * UW + ubase[g] : (a.n_kv_heads - 1 - h) * UW + h * UH + ubase[g];
  };
  const int C = static_cast<int>(U < a.L.ctas_max ? U : a.L.ctas_max);
  TreeHeader line = {};  // what next_group() needs of the header to come
  line.n_groups = n_groups;
  line.n_wide = n_wide;
  line.n_kv_heads = a.n_kv_heads;
  // No CTA has both wide and other groups: each kind gets its share of the CTAs,
  // rounded to the side that leaves the less work to the busiest one.
  const int64_t WT = WW * a.n_kv_heads;  // the wide groups' part of the line
  int CW = n_wide == n_groups ? C : 0;
  if (n_wide > 0 && n_wide < n_groups) {
    CW = static_cast<int>(min(max(C * WT / W, int64_t{1}), static_cast<int64_t>(C - 1)));
    // (rounded down a wide one has the most, WT / CW; rounded up another, (W - WT) / (C - CW - 1))
    if ((W - WT) * CW < WT * (C - CW - 1)) ++CW;
  }
  const auto cta_from = [&](int c) { return c >= C ? W : c < CW ? c * WT / CW : WT + (c - CW) * (W - WT) / (C - CW); };
  const auto cta_of = [&](int64_t w) {
    return w < WT ? cta_of_weight(w, WT, CW) : CW + cta_of_weight(w - WT, W - WT, C - CW);
  };
  // every CTA's first unit
  TreeCta *ctas = tree_at<TreeCta>(a, a.L.ctas);
  TreeCta first = {};
  for (int c = tid; c <= C && C > 0; c += kPlanThreads) {  // (C < kPlanThreads: once each)
    const int64_t lo = cta_from(c);
    if (lo >= W) {
      S.uidx[c] = U;
      continue;
    }
    const bool in_wide = lo < WT;
    const int64_t from = in_wide ? lo : lo - WT, per = in_wide ? WW : WH - WW;
    int h = static_cast<int>(from / per);
    const int64_t rem = from - h * per + (in_wide ? 0 : WW);
    int g = in_wide ? 0 : n_wide, hi = in_wide ? n_wide : n_groups;
    while (hi - g > 1) {  // the last group that starts at or before rem
      const int mid = (g + hi) >> 1;
      if (wbase[mid] <= rem) g = mid; else hi = mid;
    }
    const TreeGroup gr = groups[g];
    const TreeSpan *sp = spans + gr.span0;
    const int64_t in = rem - wbase[g];
    int s = 0;
    hi = gr.n_spans;
    while (hi - s > 1) {
      const int mid = (s + hi) >> 1;
      if (span_weight(cost, gr, mid, sp[mid].tile0) <= in) s = mid; else hi = mid;
    }
    const int64_t x = in - span_weight(cost, gr, s, sp[s].tile0);
    const int own = span_cost(cost, gr, s), tw = gr.n_cols > 128 ? cost.tile2 : cost.tile1;
    int t = x == 0 ? 0 : x <= own + tw ? 1 : static_cast<int>((x - own + tw - 1) / tw);
    if (t >= (sp[s].len + TL - 1) / TL) {
      t = 0;
      if (++s == gr.n_spans) {
        s = 0;
        next_group(line, h, g);
      }
    }
    S.uidx[c] = h < a.n_kv_heads ? units_before(h, g) + spans[groups[g].span0 + s].tile0 + t : U;
    first.head = h;
    first.group = g;
    first.span = s;
    first.tile = t;
  }
  __syncthreads();
  // a share without a unit gets no CTA: those with units are numbered anew
  const int n_units = tid < C ? static_cast<int>(S.uidx[tid + 1] - S.uidx[tid]) : 0;
  const int number = static_cast<int>(block_scan(S, n_units > 0));
  const int n_ctas = static_cast<int>(S.carry);
  if (n_units > 0) {
    first.n_units = n_units;
    first.wide = first.group < n_wide;
    first.g = groups[first.group];
    first.sp = spans[first.g.span0 + first.span];
    ctas[number] = first;
    S.number[tid] = static_cast<int16_t>(number);
  }
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  // every group's columns by 32, for the merge
  for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    const int nb = g < n_groups ? (groups[g].n_cols + 31) / 32 : 0;
    const int64_t at = block_scan(S, nb);
    for (int x = 0; x < nb; ++x) tree_at<int2>(a, a.L.blocks)[at + x] = make_int2(g, 32 * x);
  }
  const int n_col_blocks = static_cast<int>(S.carry);
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  // the records of every (kv head, group); on the tensor cores a CTA with two
  // units or more may leave two of a group with up to 128 columns (tree_tc.cu)
  const int streams = a.L.cols > 128 && U > a.L.ctas_max ? 2 : 1;
  int32_t *piece_row = tree_at<int32_t>(a, a.L.piece_row);
  int2 *piece_cta = tree_at<int2>(a, a.L.piece_cta);
  const int64_t K = C > 0 ? static_cast<int64_t>(n_groups) * a.n_kv_heads : 0;
  for (int64_t k0 = 0; k0 < K; k0 += kPlanThreads) {
    const int64_t k = k0 + tid;
    int64_t rows = 0;
    int2 pc = make_int2(0, 0);
    if (k < K) {
      const int g = static_cast<int>(k % n_groups);
      const TreeGroup gr = groups[g];
      const TreeSpan last = spans[gr.span0 + gr.n_spans - 1];
      const int64_t w = weight_before(static_cast<int>(k / n_groups), g);
      const int tiles = (last.len + TL - 1) / TL;
      pc.x = S.number[cta_of(w)];
      const int ls = gr.n_spans - 1;
      int64_t end = w + span_weight(cost, gr, ls, last.tile0);  // where the group's last unit starts
      if (tiles > 1) end += span_cost(cost, gr, ls) + static_cast<int64_t>(tiles - 1) * (gr.n_cols > 128 ? cost.tile2 : cost.tile1);
      pc.y = S.number[cta_of(end)] - pc.x + 1;
      if (streams == 2 && gr.n_cols <= 128) pc.y *= 2;
      rows = static_cast<int64_t>(pc.y) * gr.n_cols;
    }
    const int64_t at = block_scan(S, rows);
    if (k < K) {
      piece_row[k] = static_cast<int32_t>(at);
      piece_cta[k] = pc;
    }
  }
  if (tid == 0)
    hdr = TreeHeader{kTreeMagic, R, T, a.n_q_heads, a.n_kv_heads, a.head_dim, a.n_blocks, V, a.dtype,
                     n_groups, n_ctas, streams, n_col_blocks, n_wide, a.capacity, a.rope_theta};
}

// cos and sin of a position's angle for one pair: the angle in turns is exact in 64-bit integers (rope_cos_sin); here
// only what is left of the nearest quarter turn, at most an eighth, is
// rounded to fp32, so both are good to about an ulp.
__device__ __forceinline__ void rope_cos_sin_exact(int64_t rel, uint64_t phase, float *c, float *s) {
  const uint64_t turns = static_cast<uint64_t>(rel) * phase;
  const uint64_t quarter = (turns + (1ull << 61)) >> 62;
  const int64_t rest = static_cast<int64_t>(turns - (quarter << 62));
  float x, y;
  sincospif(static_cast<float>(rest) * 0x1p-63f, &y, &x);
  *c = (quarter & 1) ? ((quarter & 2) ? y : -y) : ((quarter & 2) ? -x : x);
  *s = (quarter & 1) ? ((quarter & 2) ? -x : x) : ((quarter & 2) ? -y : y);
}

// The tables: the columns of every group, and every row's rotations.
__global__ void __launch_bounds__(256) tree_tables_kernel(const __grid_constant__ TreeArgs a,
                                                          const __grid_constant__ TreeMeta m) {
  if (!tree_plan_ok(a)) return;
  const int G = a.n_q_heads / a.n_kv_heads, half = a.head_dim / 2, V = a.n_view, T = a.max_nodes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t *n_nodes = tree_at<int32_t>(a, a.L.n_nodes), *first = tree_at<int32_t>(a, a.L.col);
  const int32_t *rot0 = tree_at<int32_t>(a, a.L.rot0), *rank = tree_at<int32_t>(a, a.L.rank);
  for (int gi = blockIdx.x; gi < tree_at<TreeHeader>(a, a.L.hdr)->n_groups; gi += gridDim.x) {
    const TreeGroup g = tree_at<TreeGroup>(a, a.L.groups)[gi];
    for (int x = threadIdx.x; x < g.n_cols; x += 256) {
      int lo = g.row0, hi = g.row1 + 1;  // the last row that starts at or before the column
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= g.col0 + x) lo = mid; else hi = mid;
      }
      const int local = g.col0 + x - first[lo], i = local / G;
      tree_at<TreeColumn>(a, a.L.columns)[g.col0 + x] =
          TreeColumn{lo * T + i, local % G, rot0[lo] + i, static_cast<uint16_t>(n_nodes[lo]),
                     static_cast<uint16_t>(rank[lo] - g.rank0)};
    }
  }
  // rotations: a warp a (view entry or tree, node), a CTA a share of a row's
  const int64_t work = static_cast<int64_t>(a.n_rows) * (V + 1);
  for (int64_t x = blockIdx.x; x < work; x += gridDim.x) {
    const int r = static_cast<int>(x / (V + 1)), v = static_cast<int>(x % (V + 1)), n = n_nodes[r];
    if (n == 0 || (v < V && (m.view_block[r * V + v] < 0))) continue;
    const int64_t root = v < V ? static_cast<int64_t>(m.q_pos[r]) - m.view_offset[r * V + v]
                               : tree_at<int32_t>(a, a.L.pos)[r];
    for (int i = warp; i < n; i += 8) {
      const int64_t rel = root + tree_at<int32_t>(a, a.L.depth)[static_cast<int64_t>(r) * T + i];
      const int64_t row = (rot0[r] + static_cast<int64_t>(v) * n + i) * half;
      for (int j = lane; j < half; j += 32) {
        float2 x;
        rope_cos_sin_exact(rel, a.phase[j], &x.x, &x.y);
        tree_at<float2>(a, a.L.rot)[row + j] = x;
        if (a.L.cols > 32 && a.dtype == HW_BF16) tree_at<float2>(a, a.L.turns)[row + turn_at(j, half, 2)] = x;
        else if (a.L.cols > 32) tree_at<__half2>(a, a.L.turns)[row + turn_at(j, half, 4)] = __floats2half2_rn(x.x, x.y);
      }
    }
  }
}

// ---------------------------------------------------------------- append

// The drafted tokens written into the cache, a warp a (row, node, kv head):
//   K[h][slot + i] = rho(k_new[r][i][h], pos + depth(i)),  V = v_new
// rotated in fp32 and rounded once to the cache's type (E4M3: divided by the
// head's scale first, saturating at 448).
template <typename T, bool kFp8>
__global__ void __launch_bounds__(256) tree_append_kernel(const __grid_constant__ TreeArgs a) {
  // Dependents start only once everything before this launch is complete:
  // the attention kernel counts on it.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, half = a.head_dim / 2, D = a.head_dim;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int h = static_cast<int>(item % a.n_kv_heads);
  const int64_t node = item / a.n_kv_heads;
  const int r = static_cast<int>(node / a.max_nodes), i = static_cast<int>(node % a.max_nodes);
  const int row = min(r, a.n_rows - 1);
  const int nodes = tree_at<int32_t>(a, a.L.n_nodes)[row], rot0 = tree_at<int32_t>(a, a.L.rot0)[row];
  const int64_t slot = static_cast<int64_t>(tree_at<int32_t>(a, a.L.slot)[row]) + i;
  // (without a plan the attention launch says so)
  if (!tree_plan_ok(a) || r >= a.n_rows || i >= nodes) return;
  // the keys turn as the queries do against their own tree
  const float2 *rot = tree_at<float2>(a, a.L.rot) + (rot0 + static_cast<int64_t>(a.n_view) * nodes + i) * half;
  const T *kn = reinterpret_cast<const T *>(a.k_new) + item * D;
  const T *vn = reinterpret_cast<const T *>(a.v_new) + item * D;
  const int64_t to = (h * a.capacity + slot) * D;
  const float ks = kFp8 ? a.k_scale[h] : 1.f, vs = kFp8 ? a.v_scale[h] : 1.f;
  for (int j = lane; j < half; j += 32) {
    const float2 cs = rot[j];
    const float c = cs.x, s = cs.y;
    const float x0 = to_f32<T>(kn[j]), x1 = to_f32<T>(kn[j + half]);
    const float y0 = __fmaf_rn(x0, c, -__fmul_rn(x1, s)), y1 = __fmaf_rn(x1, c, __fmul_rn(x0, s));
    if constexpr (kFp8) {
      uint8_t *k = static_cast<uint8_t *>(a.k) + to, *v = static_cast<uint8_t *>(a.v) + to;
      k[j] = __nv_cvt_float_to_fp8(y0 / ks, __NV_SATFINITE, __NV_E4M3);
      k[j + half] = __nv_cvt_float_to_fp8(y1 / ks, __NV_SATFINITE, __NV_E4M3);
      v[j] = __nv_cvt_float_to_fp8(to_f32<T>(vn[j]) / vs, __NV_SATFINITE, __NV_E4M3);
      v[j + half] = __nv_cvt_float_to_fp8(to_f32<T>(vn[j + half]) / vs, __NV_SATFINITE, __NV_E4M3);
    } else {
      T *k = static_cast<T *>(a.k) + to, *v = static_cast<T *>(a.v) + to;
      k[j] = from_f32<T>(y0);
      k[j + half] = from_f32<T>(y1);
      v[j] = vn[j];
      v[j + half] = vn[j + half];
    }
  }
}

// ----------------------------------------------------------------- merge

// Every query's records - one for every CTA (or stream) that touched its
// group - joined as
//   M = max m,  out = sum o 2^(m - M) / sum l 2^(m - M),  lse = (M + log2 l) ln 2.
// A CTA takes 32 columns of a group, one a lane, and a quarter of the head
// dimension: a warp has 8 elements of it, which lie side by side in a record
// (a load is 32 sectors of 8 lines; with a query a warp it was 16 lines for
// half as much: 17 us instead of 14.5 for two chains of 4 nodes, 57 instead of
// 51 for 4 trees of 16).  Two to eight warps share the records of every 8
// elements and join at the end, so that up to 16 (64) records cost one trip to
// memory.
template <int D, int kShares>
struct MergeShape {
  static constexpr int kChunks = D / 32;               // of 8 elements, in a quarter
  static constexpr int kThreads = kChunks * kShares * 32;
};

// Up to 8 records from j on in steps of kShares, joined to (M, L, acc).
template <int kShares>
__device__ __forceinline__ void merge_batch(const float2 *ml, const float *o, int n_cols, int64_t step, int j, int n,
                                            float &M, float &L, float (&acc)[8]) {
  constexpr int N = 8;
  float2 x[N];
  float4 v[N][2];
  // without branches: the ones past the end read the last record again, and
  // what a record without tiles (m = -inf) holds is dropped
#pragma unroll
  for (int b = 0; b < N; ++b) {
    const int64_t at = min(j + kShares * b, n - 1);
    x[b] = ml[at * n_cols];
    const float4 *src = reinterpret_cast<const float4 *>(o + at * step);
    v[b][0] = src[0];
    v[b][1] = src[1];
  }
  float top = M;
#pragma unroll
  for (int b = 0; b < N; ++b) {
    if (j + kShares * b >= n) x[b].x = -INFINITY;
    top = fmaxf(top, x[b].x);
  }
  const float old = M == -INFINITY ? 0.f : ex2(M - top);
  M = top;
  L *= old;
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
  for (int b = 0; b < N; ++b) {
    const bool use = x[b].x != -INFINITY;
    const float w = use ? ex2(x[b].x - top) : 0.f;
    const float y[8] = {v[b][0].x, v[b][0].y, v[b][0].z, v[b][0].w, v[b][1].x, v[b][1].y, v[b][1].z, v[b][1].w};
    L = use ? fmaf(w, x[b].y, L) : L;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = use ? fmaf(w, y[e], acc[e]) : acc[e];
  }
}

template <typename T, int D, int kShares>
__global__ void __launch_bounds__(MergeShape<D, kShares>::kThreads) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kChunks = MergeShape<D, kShares>::kChunks, kRow = kChunks * 8;  // elements of a row here
  constexpr int kPiece = 16 / sizeof(T);                               // elements of a 16-byte store
  __shared__ float part[kShares][kChunks][8][32], part_m[kShares][kChunks][32], part_l[kShares][kChunks][32];
  __shared__ __align__(16) T tile[32][kRow];
  __shared__ int32_t out_row[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, chunk = warp / kShares, share = warp % kShares;
  const int quarter = blockIdx.x & 3, h = (blockIdx.x >> 2) % a.n_kv_heads, b = (blockIdx.x >> 2) / a.n_kv_heads;
  const int G = a.n_q_heads / a.n_kv_heads;
  // (loads that do not hang on one another first: trips to L2 are what this
  // kernel takes)
  const TreeHeader &hdr = *tree_at<const TreeHeader>(a, a.L.hdr);
  const int2 at = tree_at<int2>(a, a.L.blocks)[b];
  const int hq_of = tree_at<int32_t>(a, a.L.heads)[h * G + min(lane, G - 1)];
  if (!tree_plan_ok(a) || b >= hdr.n_col_blocks) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // whoever follows this grid follows that one
    return;
  }
  const TreeGroup g = tree_at<TreeGroup>(a, a.L.groups)[at.x];
  const int64_t k = static_cast<int64_t>(h) * hdr.n_groups + at.x;
  const int n = tree_at<int2>(a, a.L.piece_cta)[k].y;
  const int64_t row0 = tree_at<int32_t>(a, a.L.piece_row)[k];
  const bool on = at.y + lane < g.n_cols;
  const int col = min(at.y + lane, g.n_cols - 1);
  const TreeColumn tc = tree_at<TreeColumn>(a, a.L.columns)[g.col0 + col];
  const int hq = __shfl_sync(0xffffffffu, hq_of, tc.head);
  const float2 *ml = tree_at<float2>(a, a.L.ml) + row0 + col;
  const float *o = tree_at<float>(a, a.L.o) + record_at(row0, g.n_cols, col, (quarter * kChunks + chunk) * 8, D);
  const int64_t step = static_cast<int64_t>(g.n_cols) * D;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the records
  float M = -INFINITY, L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = share; j < n; j += 8 * kShares) merge_batch<kShares>(ml, o, g.n_cols, step, j, n, M, L, acc);
  if (share > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[share][chunk][e][lane] = acc[e];
    part_m[share][chunk][lane] = M;
    part_l[share][chunk][lane] = L;
  }
  if (tid < 32) out_row[lane] = on ? tc.node * a.n_q_heads + hq : -1;
  __syncthreads();
  if (share == 0) {
    float top = M;
#pragma unroll
    for (int x = 1; x < kShares; ++x) top = fmaxf(top, part_m[x][chunk][lane]);
    const float w0 = M == -INFINITY ? 0.f : ex2(M - top);
    L *= w0;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= w0;
#pragma unroll
    for (int x = 1; x < kShares; ++x) {
      const float m = part_m[x][chunk][lane], w = m == -INFINITY ? 0.f : ex2(m - top);
      L = fmaf(part_l[x][chunk][lane], w, L);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(part[x][chunk][e][lane], w, acc[e]);
    }
    const float inv = 1.f / L;  // (a node attends itself; NaN where its values are)
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[lane][chunk * 8 + e] = from_f32<T>(acc[e] * inv);
    if (a.lse && warp == 0 && quarter == 0 && on)
      a.lse[tc.node * a.n_q_heads + hq] = (top + log2f(L)) * 0.693147180559945309f;
  }
  __syncthreads();
  for (int x = tid; x < 32 * kRow / kPiece; x += MergeShape<D, kShares>::kThreads) {
    const int r = x / (kRow / kPiece), e = x % (kRow / kPiece) * kPiece;
    if (out_row[r] < 0) continue;
    T res[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) res[i] = tile[r][e + i];
    store_row_part<T, kPiece>(static_cast<T *>(a.out) + static_cast<int64_t>(out_row[r]) * D + quarter * kRow + e, res);
  }
}

// ---------------------------------------------------------------- commit

// The n nodes that a row of `nodes` nodes may keep: ascending node numbers.
__device__ bool path_ok(const int32_t *path, int n, int nodes) {
  bool ok = n <= nodes;
  for (int j = 0, before = -1; ok && j < n; before = path[j++]) ok = path[j] > before && path[j] < nodes;
  return ok;
}

// The accepted path of each row moved behind its block, bit for bit:
//   K[l][h][end + j] = K[l][h][slot + path[j]],  V alike,  j < n_path.
// (64 layers of 4 rows: 6.5 to 7.5 us, the call's own time on the host; 36 layers of
// 64 rows of E4M3 codes: 16 us, 4.1 TB/s of 128-byte pieces.)
// A warp moves one (layer, head, pool) line of one row in steps of ascending
// j: a destination never lies behind its own source (path[j] >= j, and the
// nodes' slots lie at or behind the block's end), so a step's stores
// overwrite only slots that steps up to it have read.
__global__ void __launch_bounds__(256) tree_commit_kernel(const __grid_constant__ TreeArgs a,
                                                          const __grid_constant__ TreeCommitArgs c) {
  __shared__ int32_t path[kMaxNodes];
  __shared__ int bad;
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  int32_t *err = reinterpret_cast<int32_t *>(a.ws);
  if (tid == 0) bad = 0;
  if (!tree_plan_ok(a)) {
    if (tid == 0) flag_error(err, HW_DEV_BAD_PLAN);
    return;
  }
  __syncthreads();
  const int32_t *n_nodes = tree_at<int32_t>(a, a.L.n_nodes);
  const int nodes = n_nodes[r], n = c.n_path[r];
  if (n == 0) return;
  const int32_t *slot_of = tree_at<int32_t>(a, a.L.slot), *end_of = tree_at<int32_t>(a, a.L.end);
  if (n < 0 || n > nodes) {
    if (tid == 0) flag_error(err, HW_DEV_BAD_TREE);
    return;
  }
  const int64_t slot = slot_of[r], end = end_of[r];
  for (int j = tid; j < n; j += blockDim.x) {
    const int p = c.path[static_cast<int64_t>(r) * a.max_nodes + j];
    const int before = j > 0 ? c.path[static_cast<int64_t>(r) * a.max_nodes + j - 1] : -1;
    if (p <= before || p >= nodes) atomicOr(&bad, 1);  // ascending node numbers
    path[j] = p;
  }
  // the destination: inside the pool, behind no other row's tokens, and
  // meeting its own row's slots only from in front
  if (tid == 0 && (end + n > a.capacity || (slot < end && slot + nodes > end))) atomicOr(&bad, 2);
  for (int x = tid; x < a.n_blocks; x += blockDim.x)
    if (ranges_meet(end, n, tree_at<int32_t>(a, a.L.block_start)[x], tree_at<int32_t>(a, a.L.block_len)[x]))
      atomicOr(&bad, 2);
  for (int x = tid; x < a.n_rows; x += blockDim.x)
    if (x != r && n_nodes[x] > 0 &&
        (ranges_meet(end, n, slot_of[x], n_nodes[x]) ||
         // (a row whose path is refused has no destination)
         (ranges_meet(end, n, end_of[x], c.n_path[x]) &&
          path_ok(c.path + static_cast<int64_t>(x) * a.max_nodes, c.n_path[x], n_nodes[x]))))
      atomicOr(&bad, 2);
  __syncthreads();
  if (bad) {
    if (tid == 0) flag_error(err, bad & 1 ? HW_DEV_BAD_TREE : HW_DEV_BAD_RANGE);
    return;
  }
  const int row_bytes = a.head_dim * c.elem_bytes, per = row_bytes / 16;  // 16-byte pieces a token: 4 .. 32
  const int64_t lines = 2ll * c.n_layers * a.n_kv_heads;
  const int span = 32 / per;  // tokens a step of the warp moves
  const int piece = lane % per;
  for (int64_t line = static_cast<int64_t>(blockIdx.x) * 8 + (tid >> 5); line < lines; line += static_cast<int64_t>(gridDim.x) * 8) {
    uint8_t *pool = static_cast<uint8_t *>(line & 1 ? c.v : c.k) + (line >> 1) * a.capacity * row_bytes;
    for (int j0 = 0; j0 < n; j0 += span) {
      const int j = j0 + lane / per;
      uint4 x;
      const bool on = j < n && slot + path[j] != end + j;
      if (on) x = *reinterpret_cast<const uint4 *>(pool + (slot + path[j]) * row_bytes + piece * 16);
      __syncwarp();
      if (on) *reinterpret_cast<uint4 *>(pool + (end + j) * row_bytes + piece * 16) = x;
      __syncwarp();
    }
  }
}

}  // namespace

// A launch that may start while the one before it on the stream ends; the
// kernel waits for that one itself (griddepcontrol.wait).
template <typename... P, typename... A>
static cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, int threads, cudaStream_t s, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_tree_plan(const TreeArgs &a, const TreeMeta &m, cudaStream_t s) {
  static bool configured = false;
  if (!configured) {
    const cudaError_t e = cudaFuncSetAttribute(tree_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(TreePlanSmem)));
    if (e != cudaSuccess) return e;
    configured = true;
  }
  tree_plan_kernel<<<1, kPlanThreads, sizeof(TreePlanSmem), s>>>(a, m);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t work = static_cast<int64_t>(a.n_rows) * (a.n_view + 1), most = 4ll * a.L.ctas_max;
  tree_tables_kernel<<<static_cast<unsigned>(work < most ? work : most), 256, 0, s>>>(a, m);
  return cudaGetLastError();
}

cudaError_t launch_tree_append(const TreeArgs &a, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(a.n_rows) * a.max_nodes * a.n_kv_heads;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8);
  if (a.dtype == HW_F32) return launch_dependent(tree_append_kernel<float, false>, grid, 256, s, a);
  if (a.dtype == HW_FP8_E4M3) return launch_dependent(tree_append_kernel<__nv_bfloat16, true>, grid, 256, s, a);
  return launch_dependent(tree_append_kernel<__nv_bfloat16, false>, grid, 256, s, a);
}

template <typename T, int D>
static cudaError_t launch_merge(const TreeArgs &a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(4 * a.n_kv_heads * a.L.max_blocks);
  // Few columns have many records each and leave most of the GPU idle: CTAs of
  // 512 threads then, whose warps share them (a layer of one tree of 2 nodes
  // over 38466 tokens, 4/2 heads: 31.2 -> 24.6 us, with head_dim 64 45 -> 32;
  // a chain of 4 over 16384, 40/8 heads: 24.8 -> 22.3).  Where the columns fill
  // the GPU two warps are enough (4 trees of 16 nodes: 38.4 us, with four 44.4).
  constexpr int kMost = 512 / D;  // a CTA of 512 threads
  return grid <= 2u * device_sm_count()
             ? launch_dependent(tree_merge_kernel<T, D, kMost>, grid, MergeShape<D, kMost>::kThreads, s, a)
             : launch_dependent(tree_merge_kernel<T, D, 2>, grid, MergeShape<D, 2>::kThreads, s, a);
}
cudaError_t launch_tree_merge(const TreeArgs &a, cudaStream_t s) {
  const bool d64 = a.head_dim == 64;
  if (a.dtype == HW_F32) return d64 ? launch_merge<float, 64>(a, s) : launch_merge<float, 128>(a, s);
  return d64 ? launch_merge<__nv_bfloat16, 64>(a, s) : launch_merge<__nv_bfloat16, 128>(a, s);
}

cudaError_t launch_tree_commit(const TreeArgs &a, const TreeCommitArgs &c, cudaStream_t s) {
  // a warp a line; many rows share the GPU, few spread out over it
  const int64_t lines = 2ll * c.n_layers * a.n_kv_heads;
  int64_t per = (lines + 7) / 8;
  const int sms = device_sm_count();
  const int64_t cap = (static_cast<int64_t>(sms > 0 ? sms : 152) * 8 + a.n_rows - 1) / a.n_rows;
  if (per > cap) per = cap;
  tree_commit_kernel<<<dim3(static_cast<unsigned>(per), static_cast<unsigned>(a.n_rows)), 256, 0, s>>>(a, c);
  return cudaGetLastError();
}

TreeLayout tree_layout(const hw_attn_desc &d, int max_nodes, int sms) {
  TreeLayout L{};
  const bool tc = tree_on_tensor_cores(d.dtype, d.head_dim);
  L.cols = tc ? 256 : 32;
  L.tile = tc ? 128 : 64;
  L.ctas_max = tc ? sms : (d.head_dim == 64 ? 3 : 2) * sms;  // what fits an SM at once
  if (L.ctas_max > 1000) L.ctas_max = 1000;  // (one thread of the plan each)
  const int64_t R = d.n_rows, V = d.max_view_blocks, G = d.n_q_heads / d.n_kv_heads;
  const int64_t Q = R * max_nodes;  // nodes
  L.max_cols = Q * G;
  // a row ends a group early at most once, and is cut by each full one
  L.max_groups = R + L.max_cols / L.cols + 1;
  const int64_t parts = R + L.max_groups;  // (row, group) pairs
  L.max_spans = parts * (V + 1);
  // spans of blocks times rows: a group has up to min(R, cols) rows
  L.max_map = parts * V * (R < L.cols ? R : L.cols);
  L.max_rots = Q * (V + 1);
  L.max_rows = (d.n_kv_heads * L.max_cols + static_cast<int64_t>(L.ctas_max) * L.cols) * (tc ? 2 : 1);
  size_t at = 256;
  auto put = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  L.hdr = put(sizeof(TreeHeader));
  L.groups = put(sizeof(TreeGroup) * L.max_groups);
  L.wbase = put(2 * sizeof(int64_t) * L.max_groups);  // weights, then units before each group
  L.spans = put(sizeof(TreeSpan) * L.max_spans);
  L.map = put(2 * L.max_map);
  L.columns = put(sizeof(TreeColumn) * L.max_cols);
  L.rot = put(4 * static_cast<size_t>(d.head_dim) * L.max_rots);
  L.turns = put((!tc ? 0 : d.dtype == HW_BF16 ? 4 : 2) * static_cast<size_t>(d.head_dim) * L.max_rots);
  L.max_blocks = L.max_cols / 32 + L.max_groups;
  L.blocks = put(8 * L.max_blocks);
  L.piece_row = put(4 * L.max_groups * d.n_kv_heads);
  L.piece_cta = put(8 * L.max_groups * d.n_kv_heads);
  L.ctas = put(sizeof(TreeCta) * L.ctas_max);
  L.n_nodes = put(4 * R);
  L.slot = put(4 * R);
  L.pos = put(4 * R);
  L.end = put(4 * R);
  L.col = put(4 * R);
  L.rot0 = put(4 * R);
  L.rank = put(4 * R);
  L.depth = put(4 * Q);
  L.mask = put(16 * Q);
  L.heads = put(4 * d.n_q_heads);
  L.block_start = put(4 * static_cast<size_t>(d.n_blocks));
  L.block_len = put(4 * static_cast<size_t>(d.n_blocks));
  L.ml = put(8 * L.max_rows);
  L.o = put(4 * static_cast<size_t>(d.head_dim) * L.max_rows);
  L.total = at;
  return L;
}

}  // namespace hw
