// tree_plan.cu - the draft-tree operators' plan (hw_tree.h), the write of the
// drafted tokens into the cache, the merge of the partial results, and the
// commit of an accepted path.
#include <cuda_fp8.h>

#include "hw_device.cuh"
#include "hw_tree.h"

namespace hw {

namespace {

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Weights of the unit line.  Tensor cores: a tile against up to 128 columns
// is bound by its K/V bytes, one against 129..256 by both products and the
// softmax of two query tiles; a segment costs its queries and its records.
struct TreeCost {
  int32_t tile1, tile2, seg;
};
__host__ __device__ inline TreeCost tree_cost(int cols) {
  return cols > 128 ? TreeCost{2, 3, 3} : TreeCost{2, 2, 1};
}

struct TreePlanSmem {
  int32_t len[HW_MAX_BLOCKS], start[HW_MAX_BLOCKS];
  int32_t refs[HW_MAX_BLOCKS + 1], cols[HW_MAX_BLOCKS], seg0[HW_MAX_BLOCKS + 1];
  int64_t scan[kPlanWarps + 1];
  int64_t carry;
  int64_t uidx[1025];
  int32_t ok;
  uint8_t parent[kPlanWarps][kMaxNodes];
  int16_t vb[HW_MAX_VIEW_ENTRIES];    // block of every view entry, -1: none
  uint8_t nodes[HW_MAX_VIEW_ENTRIES];  // nodes of every row (rows <= HW_MAX_VIEW_ENTRIES)
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

// One row, by one warp: its checks, depths and ancestor masks.  Returns its
// node count (0 if the row is refused).
__device__ int plan_row(const TreeArgs &a, const TreeMeta &m, TreePlanSmem &S, int32_t *err, int r,
                        int lane) {
  const int T = a.max_nodes, R = a.n_rows;
  int n = m.n_nodes[r];
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
  // the nodes' tokens: inside the pool, outside every block and other tree
  const int64_t slot = tree_slot(m, a.n_blocks, r);
  bool bad_range = S.len[b] < 0 || slot < 0 || slot + n > a.capacity;
  for (int x = lane; x < a.n_blocks; x += 32)
    bad_range |= ranges_meet(slot, n, S.start[x], S.len[x]);
  for (int x = lane; x < R; x += 32)
    if (x != r) bad_range |= ranges_meet(slot, n, tree_slot(m, a.n_blocks, x), m.n_nodes[x]);
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

// Weight before tile t of a segment (t > 0 includes the segment's own).
__device__ __forceinline__ int64_t tile_weight(const TreeCost &c, int n_cols, int t) {
  return t == 0 ? 0 : c.seg + static_cast<int64_t>(t) * (n_cols > 128 ? c.tile2 : c.tile1);
}
// The CTA that owns a unit starting at weight w.
__device__ __forceinline__ int cta_of_weight(int64_t w, int64_t W, int C) {
  return static_cast<int>(((w + 1) * C - 1) / W);
}

// The whole plan, by one CTA.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const __grid_constant__ TreeArgs a,
                                                                 const __grid_constant__ TreeMeta m) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  TreePlanSmem &S = *reinterpret_cast<TreePlanSmem *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.n_rows, V = a.n_view, E = R * V, T = a.max_nodes;
  const int G = a.n_q_heads / a.n_kv_heads, CG = a.L.cols;
  const TreeCost cost = tree_cost(CG);
  int32_t *err = reinterpret_cast<int32_t *>(a.ws);
  TreeHeader &hdr = *tree_at<TreeHeader>(a, a.L.hdr);
  int32_t *n_nodes = tree_at<int32_t>(a, a.L.n_nodes);
  int32_t *entry_seg = tree_at<int32_t>(a, a.L.entry_seg), *entry_col = tree_at<int32_t>(a, a.L.entry_col);
  TreeRef *refs = tree_at<TreeRef>(a, a.L.refs);
  TreeSeg *segs = tree_at<TreeSeg>(a, a.L.segs);
  int64_t *wbase = tree_at<int64_t>(a, a.L.wbase);
  if (tid == 0) {
    S.ok = 1;
    S.carry = 0;
    hdr.magic = 0;
  }
  // blocks: the usable length of each (0: skipped)
  for (int b = tid; b < a.n_blocks; b += kPlanThreads) {
    const int st = m.block_start[b], ln = m.block_len[b];
    const bool bad = st < 0 || ln < 0 || static_cast<int64_t>(st) + ln > a.capacity;
    if (bad) flag_error(err, HW_DEV_BAD_RANGE);
    S.start[b] = bad ? 0 : st;
    S.len[b] = bad ? -1 : ln;
    tree_at<int32_t>(a, a.L.block_start)[b] = S.start[b];
    tree_at<int32_t>(a, a.L.block_len)[b] = S.len[b];
    S.refs[b] = 0;
    S.cols[b] = 0;
  }
  __syncthreads();
  for (int r = warp; r < R; r += kPlanWarps) {
    const int n = plan_row(a, m, S, err, r, lane);
    if (lane == 0) {
      n_nodes[r] = n;
      S.nodes[r] = static_cast<uint8_t>(n);
    }
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
  for (int e = tid; e < E; e += kPlanThreads) {
    const int b = m.view_block[e];
    const bool bad = b < -1 || b >= a.n_blocks;
    if (bad) flag_error(err, HW_DEV_BAD_BLOCK);
    S.vb[e] = static_cast<int16_t>(bad ? -1 : b);
    entry_seg[e] = -1;
    entry_col[e] = 0;
  }
  __syncthreads();
  if (!S.ok) {  // no usable head map: the plan attends and writes nothing
    for (int r = tid; r < R; r += kPlanThreads) {
      n_nodes[r] = 0;
      S.nodes[r] = 0;
    }
    __syncthreads();
  }
  // references of every block: first counted, then written in entry order
  for (int pass = 0; pass < 2; ++pass) {
    for (int b = warp; b < a.n_blocks; b += kPlanWarps) {
      int nref = 0, ncol = 0;
      if (S.len[b] > 0) {
        for (int e0 = 0; e0 < E; e0 += 32) {
          const int e = e0 + lane;
          const int r = e < E ? e / V : 0;
          const int n = e < E && S.vb[e] == b ? S.nodes[r] : 0;
          const unsigned hit = __ballot_sync(0xffffffffu, n > 0);
          if (!hit) continue;
          int incl = n * G;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          if (pass && n > 0) {
            TreeRef ref;
            ref.row = r;
            ref.col = ncol + incl - n * G;
            ref.rel = static_cast<int64_t>(m.q_pos[r]) - m.view_offset[e];
            refs[S.refs[b] + nref + __popc(hit & lanemask_lt(lane))] = ref;
            entry_seg[e] = S.seg0[b];
            entry_col[e] = ref.col;
          }
          nref += __popc(hit);
          ncol += __shfl_sync(0xffffffffu, incl, 31);
        }
      }
      if (!pass && lane == 0) {
        S.refs[b] = nref;
        S.cols[b] = ncol;
      }
      if (pass) {
        const int first = S.refs[b], seg0 = S.seg0[b];
        for (int g = lane; g * CG < ncol; g += 32)
          segs[seg0 + g] = TreeSeg{S.start[b], S.len[b], -1, first, nref, g * CG, min(CG, ncol - g * CG), 0, 0, {}};
      }
    }
    __syncthreads();
    if (!pass && tid == 0) {
      int ref0 = 0, seg0 = 0;
      for (int b = 0; b < a.n_blocks; ++b) {
        const int nr = S.refs[b];
        S.refs[b] = ref0;
        S.seg0[b] = seg0;
        ref0 += nr;
        seg0 += (S.cols[b] + CG - 1) / CG;
      }
      S.seg0[a.n_blocks] = seg0;
      S.carry = seg0;
    }
    __syncthreads();
  }
  // the rows' trees
  for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    const int n = r < R ? n_nodes[r] : 0;
    const int ns = (n * G + CG - 1) / CG;
    const int s0 = static_cast<int>(block_scan(S, ns));
    if (r < R) {
      entry_seg[E + r] = n > 0 ? s0 : -1;
      entry_col[E + r] = 0;
      refs[E + r] = TreeRef{r, 0, n > 0 ? tree_at<int32_t>(a, a.L.pos)[r] : 0};
      const int at = n > 0 ? tree_at<int32_t>(a, a.L.slot)[r] : 0;
      for (int g = 0; g < ns; ++g)
        segs[s0 + g] = TreeSeg{at, n, r, E + r, 1, g * CG, min(CG, n * G - g * CG), 0, 0, {}};
    }
  }
  const int n_segs = static_cast<int>(S.carry);
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  // the weighted line, and (in the high half) the units before each segment
  const int TL = a.L.tile;
  for (int s0 = 0; s0 < n_segs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t w = 0;
    if (s < n_segs) w = tile_weight(cost, segs[s].n_cols, (segs[s].len + TL - 1) / TL);
    const int64_t at = block_scan(S, w);
    if (s < n_segs) wbase[s] = at;
  }
  const int64_t WH = S.carry, W = WH * a.n_kv_heads;
  const int64_t most = W / (cost.seg + cost.tile2);
  const int C = static_cast<int>(most < a.L.ctas_max ? most : a.L.ctas_max);
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  // the segments' places in the column table
  for (int s0 = 0; s0 < n_segs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const int64_t at = block_scan(S, s < n_segs ? segs[s].n_cols : 0);
    if (s < n_segs) {
      segs[s].table = static_cast<int32_t>(at);
      // (a block's columns are whole groups of G: its first one starts a row)
      segs[s].rot0 = static_cast<int32_t>((at - segs[s].col0) / G);
    }
  }
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  int64_t *ubase = wbase + a.L.max_segs;
  for (int s0 = 0; s0 < n_segs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const int64_t at = block_scan(S, s < n_segs ? (segs[s].len + TL - 1) / TL : 0);
    if (s < n_segs) ubase[s] = at;
  }
  const int64_t UH = S.carry;
  __syncthreads();
  if (tid == 0) S.carry = 0;
  __syncthreads();
  // every CTA's first unit
  TreeCta *ctas = tree_at<TreeCta>(a, a.L.ctas);
  for (int c = tid; c <= C && C > 0; c += kPlanThreads) {
    const int64_t lo = c * W / C;
    int h = static_cast<int>(lo / WH), s = 0, t = 0;
    if (h >= a.n_kv_heads) {
      S.uidx[c] = UH * a.n_kv_heads;
      continue;
    }
    const int64_t rem = lo - h * WH;
    int hi = n_segs;
    while (hi - s > 1) {  // the last segment that starts at or before rem
      const int mid = (s + hi) >> 1;
      if (wbase[mid] <= rem) s = mid; else hi = mid;
    }
    const int64_t in = rem - wbase[s];
    const int tw = segs[s].n_cols > 128 ? cost.tile2 : cost.tile1;
    const int tiles = (segs[s].len + TL - 1) / TL;
    if (in > 0) t = in <= cost.seg + tw ? 1 : static_cast<int>((in - cost.seg + tw - 1) / tw);
    if (t >= tiles) {
      t = 0;
      if (++s == n_segs) {
        s = 0;
        ++h;
      }
    }
    S.uidx[c] = h < a.n_kv_heads ? h * UH + ubase[s] + t : UH * a.n_kv_heads;
    if (c < C) ctas[c] = TreeCta{h, s, t, 0};
  }
  __syncthreads();
  for (int c = tid; c < C; c += kPlanThreads) ctas[c].n_units = static_cast<int>(S.uidx[c + 1] - S.uidx[c]);
  // the records of every (kv head, segment)
  int32_t *piece_row = tree_at<int32_t>(a, a.L.piece_row);
  int2 *piece_cta = tree_at<int2>(a, a.L.piece_cta);
  const int64_t K = C > 0 ? static_cast<int64_t>(n_segs) * a.n_kv_heads : 0;
  for (int64_t k0 = 0; k0 < K; k0 += kPlanThreads) {
    const int64_t k = k0 + tid;
    int64_t rows = 0;
    int2 pc = make_int2(0, 0);
    if (k < K) {
      const int h = static_cast<int>(k / n_segs), s = static_cast<int>(k % n_segs);
      const int tiles = (segs[s].len + TL - 1) / TL;
      const int64_t w = h * WH + wbase[s];
      pc.x = cta_of_weight(w, W, C);
      pc.y = cta_of_weight(w + tile_weight(cost, segs[s].n_cols, tiles - 1), W, C) - pc.x + 1;
      rows = static_cast<int64_t>(pc.y) * segs[s].n_cols;
    }
    const int64_t at = block_scan(S, rows);
    if (k < K) {
      piece_row[k] = static_cast<int32_t>(at);
      piece_cta[k] = pc;
    }
  }
  if (tid == 0)
    hdr = TreeHeader{kTreeMagic, R, T, a.n_q_heads, a.n_kv_heads, a.head_dim, a.n_blocks, V, a.dtype,
                     n_segs, C, 0, a.capacity};
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

// The columns' queries, a CTA a segment, and their rotations, a warp a row.
__global__ void __launch_bounds__(256) tree_columns_kernel(const __grid_constant__ TreeArgs a) {
  if (!tree_plan_ok(a)) return;
  const int n_segs = tree_at<TreeHeader>(a, a.L.hdr)->n_segs;
  const int G = a.n_q_heads / a.n_kv_heads, half = a.head_dim / 2;
  const int lane = threadIdx.x & 31;
  const TreeRef *refs = tree_at<TreeRef>(a, a.L.refs);
  for (int s = blockIdx.x; s < n_segs; s += gridDim.x) {
    const TreeSeg sg = tree_at<TreeSeg>(a, a.L.segs)[s];
    auto ref_of = [&](int col) {
      int lo = 0, hi = sg.n_ref;  // the reference that holds the column
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (refs[sg.ref0 + mid].col <= col) lo = mid; else hi = mid;
      }
      return refs[sg.ref0 + lo];
    };
    for (int x = threadIdx.x; x < sg.n_cols; x += 256) {
      const int col = sg.col0 + x;
      const TreeRef ref = ref_of(col);
      const int local = col - ref.col;
      tree_at<TreeColumn>(a, a.L.columns)[sg.table + x] =
          TreeColumn{ref.row * a.max_nodes + local / G, local % G, sg.rot0 + col / G, 0};
    }
    // rows whose first column is the segment's
    const int p0 = (sg.col0 + G - 1) / G, p1 = (sg.col0 + sg.n_cols + G - 1) / G;
    for (int p = p0 + (threadIdx.x >> 5); p < p1; p += 8) {
      const TreeRef ref = ref_of(p * G);
      const int64_t rel = ref.rel + tree_at<int32_t>(a, a.L.depth)[ref.row * a.max_nodes + p - ref.col / G];
      float2 *to = tree_at<float2>(a, a.L.rot) + static_cast<int64_t>(sg.rot0 + p) * half;
      for (int j = lane; j < half; j += 32) rope_cos_sin_exact(rel, a.phase[j], &to[j].x, &to[j].y);
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
  if (!tree_plan_ok(a)) return;  // the attention launch records it
  const int lane = threadIdx.x & 31, half = a.head_dim / 2, D = a.head_dim;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int h = static_cast<int>(item % a.n_kv_heads);
  const int64_t node = item / a.n_kv_heads;
  const int r = static_cast<int>(node / a.max_nodes), i = static_cast<int>(node % a.max_nodes);
  if (r >= a.n_rows || i >= tree_at<int32_t>(a, a.L.n_nodes)[r]) return;
  // the tree's own segment holds the keys' rotations too
  const TreeSeg &sg = tree_at<TreeSeg>(a, a.L.segs)[tree_at<int32_t>(a, a.L.entry_seg)[a.n_rows * a.n_view + r]];
  const float2 *rot = tree_at<float2>(a, a.L.rot) + static_cast<int64_t>(sg.rot0 + i) * half;
  const int64_t slot = static_cast<int64_t>(tree_at<int32_t>(a, a.L.slot)[r]) + i;
  const T *kn = reinterpret_cast<const T *>(a.k_new) + item * D;
  const T *vn = reinterpret_cast<const T *>(a.v_new) + item * D;
  const int64_t to = (h * a.capacity + slot) * D;
  const float ks = kFp8 ? a.k_scale[h] : 1.f, vs = kFp8 ? a.v_scale[h] : 1.f;
  for (int j = lane; j < half; j += 32) {
    const float c = rot[j].x, s = rot[j].y;
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

constexpr int kMergeWarps = 8;
constexpr int kMergeList = 256;  // records a warp lists at a time

// One (row, node, q head) a warp: its records - one for every CTA that
// touched a segment holding its column - joined as
//   M = max m,  out = sum o 2^(m - M) / sum l 2^(m - M),  lse = (M + log2 l) ln 2.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int EPL = D / 32;
  __shared__ int2 list_s[kMergeWarps][kMergeList];  // record's first row; its columns, the item's column
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!tree_plan_ok(a)) return;
  const TreeHeader &hdr = *tree_at<const TreeHeader>(a, a.L.hdr);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp;
  const int G = a.n_q_heads / a.n_kv_heads;
  const int x = static_cast<int>(item % a.n_q_heads);  // place in the head list: kv head, then its q heads
  const int64_t node = item / a.n_q_heads;
  const int r = static_cast<int>(node / a.max_nodes), i = static_cast<int>(node % a.max_nodes);
  if (r >= a.n_rows || i >= tree_at<int32_t>(a, a.L.n_nodes)[r]) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // whoever follows this grid follows that one
    return;
  }
  const int h = x / G, hq = tree_at<int32_t>(a, a.L.heads)[x];
  const int local = i * G + x % G;
  int2 *list = list_s[warp];
  bool waited = false;
  const int32_t *entry_seg = tree_at<int32_t>(a, a.L.entry_seg), *entry_col = tree_at<int32_t>(a, a.L.entry_col);
  const float2 *ml = tree_at<float2>(a, a.L.ml);
  const float *o = tree_at<float>(a, a.L.o);
  float M = -INFINITY, L = 0.f, acc[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  // usually one window: a view that names one block many times has more
  for (int first = 0, total = 1; first < total; first += kMergeList) {
    // the records' rows, from the row's view entries and its tree
    int n = 0;
    for (int v0 = 0; v0 <= a.n_view; v0 += 32) {
      const int v = v0 + lane;
      int cnt = 0, row0 = 0, step = 0, col = 0;
      if (v <= a.n_view) {
        const int e = v < a.n_view ? r * a.n_view + v : a.n_rows * a.n_view + r;
        const int s0 = entry_seg[e];
        if (s0 >= 0) {
          col = entry_col[e] + local;
          const int s = s0 + col / a.L.cols;
          col %= a.L.cols;
          const int64_t k = static_cast<int64_t>(h) * hdr.n_segs + s;
          cnt = tree_at<int2>(a, a.L.piece_cta)[k].y;
          step = tree_at<TreeSeg>(a, a.L.segs)[s].n_cols;
          row0 = tree_at<int32_t>(a, a.L.piece_row)[k];
        }
      }
      int incl = cnt;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      const int at = n + incl - cnt - first;
      for (int j = max(0, -at); j < cnt && at + j < kMergeList; ++j)
        list[at + j] = make_int2(row0 + j * step, step << 16 | col);
      n += __shfl_sync(0xffffffffu, incl, 31);
    }
    __syncwarp();
    total = n;
    n = min(n - first, kMergeList);
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the records
    waited = true;
    float top = M;
    for (int j = lane; j < n; j += 32) top = fmaxf(top, ml[list[j].x + (list[j].y & 0xffff)].x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float old = M == -INFINITY ? 0.f : ex2(M - top);
    M = top;
    L *= old;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] *= old;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const int2 at = list[j];
      const int col = at.y & 0xffff;
      const float2 x2 = ml[at.x + col];
      const float w = M == -INFINITY ? 0.f : ex2(x2.x - M);
      L += x2.y * w;
      const float *src = o + record_at(at.x, at.y >> 16, col, lane * EPL, D);
      float val[EPL];
      if constexpr (EPL == 4) {
        const float4 y = *reinterpret_cast<const float4 *>(src);
        val[0] = y.x; val[1] = y.y; val[2] = y.z; val[3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2 *>(src);
        val[0] = y.x; val[1] = y.y;
      }
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = fmaf(w, val[e], acc[e]);
    }
    __syncwarp();
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  T res[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) res[e] = from_f32<T>(acc[e] * inv);
  const int64_t out_row = node * a.n_q_heads + hq;
  store_row_part<T, EPL>(static_cast<T *>(a.out) + out_row * D + lane * EPL, res);
  if (a.lse && lane == 0)
    a.lse[out_row] = L > 0.f ? (M + log2f(L)) * 0.693147180559945309f : -INFINITY;
}

// ---------------------------------------------------------------- commit

// The accepted path of each row moved behind its block, bit for bit:
//   K[l][h][end + j] = K[l][h][slot + path[j]],  V alike,  j < n_path.
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
         ranges_meet(end, n, end_of[x], min(max(c.n_path[x], 0), n_nodes[x]))))
      atomicOr(&bad, 2);
  __syncthreads();
  if (bad) {
    if (tid == 0) flag_error(err, (bad & 1 ? HW_DEV_BAD_TREE : 0) | (bad & 2 ? HW_DEV_BAD_RANGE : 0));
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
  static_assert(sizeof(TreePlanSmem) <= 48 * 1024, "the plan's shared memory needs no opt-in");
  tree_plan_kernel<<<1, kPlanThreads, sizeof(TreePlanSmem), s>>>(a, m);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t most = 4ll * a.L.ctas_max;
  tree_columns_kernel<<<static_cast<unsigned>(a.L.max_segs < most ? a.L.max_segs : most), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_append(const TreeArgs &a, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(a.n_rows) * a.max_nodes * a.n_kv_heads;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8);
  if (a.dtype == HW_F32) return launch_dependent(tree_append_kernel<float, false>, grid, 256, s, a);
  if (a.dtype == HW_FP8_E4M3) return launch_dependent(tree_append_kernel<__nv_bfloat16, true>, grid, 256, s, a);
  return launch_dependent(tree_append_kernel<__nv_bfloat16, false>, grid, 256, s, a);
}

cudaError_t launch_tree_merge(const TreeArgs &a, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(a.n_rows) * a.max_nodes * a.n_q_heads;
  const unsigned grid = static_cast<unsigned>((items + kMergeWarps - 1) / kMergeWarps);
  const bool d64 = a.head_dim == 64;
  if (a.dtype == HW_F32)
    return launch_dependent(d64 ? tree_merge_kernel<float, 64> : tree_merge_kernel<float, 128>, grid, kMergeWarps * 32, s, a);
  return launch_dependent(d64 ? tree_merge_kernel<__nv_bfloat16, 64> : tree_merge_kernel<__nv_bfloat16, 128>, grid,
                          kMergeWarps * 32, s, a);
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
  L.ctas_max = tc ? sms : 2 * sms;
  if (L.ctas_max > 1024) L.ctas_max = 1024;
  const int64_t R = d.n_rows, E = R * d.max_view_blocks, G = d.n_q_heads / d.n_kv_heads;
  const int64_t Q = R * max_nodes;  // nodes
  const int64_t block_cols = Q * d.max_view_blocks * G, tree_cols = Q * G;
  L.max_refs = E + R;
  // sum of ceil(cols / L.cols) over the referenced blocks and the trees
  L.max_segs = d.n_blocks + block_cols / L.cols + R + tree_cols / L.cols + 1;
  L.max_cols = block_cols + tree_cols;
  L.max_rots = L.max_cols / G;
  L.max_rows = d.n_kv_heads * (block_cols + tree_cols) + static_cast<int64_t>(L.ctas_max) * L.cols;
  size_t at = 256;
  auto put = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return o;
  };
  L.hdr = put(sizeof(TreeHeader));
  L.segs = put(sizeof(TreeSeg) * L.max_segs);
  L.wbase = put(2 * sizeof(int64_t) * L.max_segs);  // weights, then units before each segment
  L.refs = put(sizeof(TreeRef) * L.max_refs);
  L.columns = put(sizeof(TreeColumn) * L.max_cols);
  L.rot = put(4 * static_cast<size_t>(d.head_dim) * L.max_rots);
  L.entry_seg = put(4 * L.max_refs);
  L.entry_col = put(4 * L.max_refs);
  L.piece_row = put(4 * L.max_segs * d.n_kv_heads);
  L.piece_cta = put(8 * L.max_segs * d.n_kv_heads);
  L.ctas = put(sizeof(TreeCta) * L.ctas_max);
  L.n_nodes = put(4 * R);
  L.slot = put(4 * R);
  L.pos = put(4 * R);
  L.end = put(4 * R);
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
