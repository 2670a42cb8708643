// cache_api.cpp - host side of the cache calls that are no attention: tokens
// written and read, commits between 4-bit caches, moves within a pool.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <numeric>

#include "hogwild.h"
#include "hw_cache.h"
#include "hw_internal.h"

namespace hw {

namespace {

bool any_misaligned(std::initializer_list<const void *> ps, uintptr_t to) {
  for (const void *p : ps)
    if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return true;
  return false;
}

// Bytes of a stored row (a token's key or value of one kv head), 0 for a
// dtype or head_dim that the cache calls do not take.
int row_bytes(int32_t dtype, int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  switch (dtype) {
    case HW_F32: return 4 * head_dim;
    case HW_BF16: return 2 * head_dim;
    case HW_FP8_E4M3: return head_dim == 128 ? 128 : 0;
    case HW_FP4_E2M1: return head_dim == 128 ? 64 : 0;
    default: return 0;
  }
}
bool known_dtype(int32_t dtype) {
  return dtype == HW_F32 || dtype == HW_BF16 || dtype == HW_FP8_E4M3 || dtype == HW_FP4_E2M1;
}

// [a, a + na) and [b, b + nb) have a token in common.
bool meets(int64_t a, int64_t na, int64_t b, int64_t nb) {
  return na > 0 && nb > 0 && a < b + nb && b < a + na;
}
bool spans_meet(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// What hw_cache_write and hw_cache_read have in common; HW_OK with *none set:
// nothing to do.
int check_cache(int32_t dtype, int32_t n_layers, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
                const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                const void *kv_scale, int64_t capacity, const int32_t *slot, const void *k, const void *v,
                bool *none) {
  *none = false;
  if (!known_dtype(dtype)) return HW_ERR_INVALID;
  if (n_layers < 0 || n_tokens < 0 || n_kv_heads <= 0 || capacity < 0) return HW_ERR_INVALID;
  if (!row_bytes(dtype, head_dim)) return HW_ERR_UNSUPPORTED;
  if (n_kv_heads > HW_MAX_Q_HEADS || capacity > INT32_MAX) return HW_ERR_UNSUPPORTED;
  if (n_layers == 0 || n_tokens == 0) {
    *none = true;
    return HW_OK;
  }
  if (!k || !v || !slot || (capacity > 0 && (!k_cache || !v_cache))) return HW_ERR_INVALID;
  if (dtype == HW_FP8_E4M3 && (!k_scale || !v_scale || any_misaligned({k_scale, v_scale}, 4))) return HW_ERR_INVALID;
  if (dtype == HW_FP4_E2M1 && capacity > 0 && !kv_scale) return HW_ERR_INVALID;
  if (any_misaligned({k_cache, v_cache, k, v}, 16) || any_misaligned({slot}, 4)) return HW_ERR_INVALID;
  if (dtype == HW_FP4_E2M1 && any_misaligned({kv_scale}, 4)) return HW_ERR_INVALID;
  return HW_OK;
}

}  // namespace

}  // namespace hw

using namespace hw;

extern "C" {

int hw_cache_write(int32_t dtype, int32_t n_layers, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
                   double rope_theta, const void *k_new, const void *v_new, const int32_t *slot,
                   const int32_t *pos, void *k_cache, void *v_cache, const float *k_scale,
                   const float *v_scale, void *kv_scale, int64_t capacity, int32_t *flags, void *stream) {
  bool none = false;
  if (!(rope_theta > 1.0) || !std::isfinite(rope_theta)) return HW_ERR_INVALID;
  const int st = check_cache(dtype, n_layers, n_tokens, n_kv_heads, head_dim, k_cache, v_cache, k_scale, v_scale,
                             kv_scale, capacity, slot, k_new, v_new, &none);
  if (st != HW_OK || none) return st;
  if (!pos || any_misaligned({pos, flags}, 4)) return HW_ERR_INVALID;
  CacheArgs a;
  std::memset(&a, 0, sizeof a);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.kv_scale = kv_scale;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_new = k_new;
  a.v_new = v_new;
  a.slot = slot;
  a.pos = pos;
  a.flags = flags;
  a.n_tokens = n_tokens;
  a.n_layers = n_layers;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.capacity = capacity;
  rope_phase_table(head_dim, rope_theta, a.phase);
  const cudaError_t e = launch_cache_write(a, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

int hw_cache_read(int32_t dtype, int32_t n_layers, int32_t n_tokens, int32_t n_kv_heads, int32_t head_dim,
                  const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                  const void *kv_scale, int64_t capacity, const int32_t *slot, void *k_out, void *v_out,
                  int32_t *flags, void *stream) {
  bool none = false;
  const int st = check_cache(dtype, n_layers, n_tokens, n_kv_heads, head_dim, k_cache, v_cache, k_scale, v_scale,
                             kv_scale, capacity, slot, k_out, v_out, &none);
  if (st != HW_OK || none) return st;
  if (any_misaligned({flags}, 4)) return HW_ERR_INVALID;
  CacheArgs a;
  std::memset(&a, 0, sizeof a);
  a.k_cache = const_cast<void *>(k_cache);
  a.v_cache = const_cast<void *>(v_cache);
  a.kv_scale = const_cast<void *>(kv_scale);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slot = slot;
  a.k_out = k_out;
  a.v_out = v_out;
  a.flags = flags;
  a.n_tokens = n_tokens;
  a.n_layers = n_layers;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.capacity = capacity;
  const cudaError_t e = launch_cache_read(a, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

int hw_block_commit_many_fp4(int32_t n_layers, int32_t n_kv_heads, int32_t head_dim, double rope_theta,
                             const void *k_src, const void *v_src, const void *scale_src, int64_t src_capacity,
                             void *k_dst, void *v_dst, void *scale_dst, int64_t dst_capacity, int32_t n_commits,
                             const int32_t *src_begin, const int32_t *n_tokens, const int32_t *dst_offset,
                             const int32_t *pos_delta, void *stream) {
  // the checks and the arguments of hw_block_commit_many, then those of the scales
  CommitArgs a;
  const int st = commit_check(HW_FP4_E2M1, n_layers, n_kv_heads, head_dim, rope_theta, k_src, v_src, src_capacity,
                              k_dst, v_dst, dst_capacity, n_commits, src_begin, n_tokens, dst_offset, pos_delta, &a);
  if (st != HW_OK || a.n_commits == 0) return st;
  if (!scale_src || !scale_dst || any_misaligned({scale_src, scale_dst}, 4)) return HW_ERR_INVALID;
  const int64_t rows = static_cast<int64_t>(n_layers) * n_kv_heads;
  const struct {
    const void *p;
    int64_t bytes;
  } to[] = {{k_dst, rows * dst_capacity * 64}, {v_dst, rows * dst_capacity * 64}},
    from[] = {{k_src, rows * src_capacity * 64}, {v_src, rows * src_capacity * 64}};
  const int64_t ns = rows * src_capacity * 4, nd = rows * dst_capacity * 4;
  for (const auto &t : to)
    if (spans_meet(t.p, t.bytes, scale_src, ns) || spans_meet(t.p, t.bytes, scale_dst, nd)) return HW_ERR_OVERLAP;
  for (const auto &f : from)
    if (spans_meet(f.p, f.bytes, scale_dst, nd)) return HW_ERR_OVERLAP;
  // One array exactly where the pools are one: codes and scales of a token would part otherwise.  (The
  // ranges are disjoint then: commit_check compares every destination with every source.)
  if (k_src == v_dst || v_src == k_dst) return HW_ERR_OVERLAP;  // (keys among values: their scales' places differ)
  const bool one_pool = k_src == k_dst || v_src == v_dst;
  if (one_pool ? k_src != k_dst || v_src != v_dst || scale_src != scale_dst || src_capacity != dst_capacity
               : spans_meet(scale_src, ns, scale_dst, nd))
    return HW_ERR_OVERLAP;
  const CommitScales scales = {static_cast<const uint32_t *>(scale_src), static_cast<uint32_t *>(scale_dst)};
  const cudaError_t e = launch_commit_fp4(a, scales, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

int hw_block_move(int32_t dtype, int32_t n_layers, int32_t n_kv_heads, int32_t head_dim, void *k_cache,
                  void *v_cache, void *kv_scale, int64_t capacity, int32_t n_moves, const int32_t *src_begin,
                  const int32_t *n_tokens, const int32_t *dst_begin, void *stream) {
  if (!known_dtype(dtype)) return HW_ERR_INVALID;
  if (n_moves < 0 || n_moves > HW_MAX_MOVES) return HW_ERR_INVALID;
  if (n_moves > 0 && (!src_begin || !n_tokens || !dst_begin)) return HW_ERR_INVALID;
  if (n_layers < 0 || n_kv_heads <= 0 || capacity < 0) return HW_ERR_INVALID;
  for (int m = 0; m < n_moves; ++m)
    if (n_tokens[m] < 0 || src_begin[m] < 0 || dst_begin[m] < 0) return HW_ERR_INVALID;
  const int row = row_bytes(dtype, head_dim);
  if (!row) return HW_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(n_layers) * n_kv_heads;
  if (rows > INT32_MAX / 4 || capacity > INT32_MAX) return HW_ERR_UNSUPPORTED;
  MoveArgs a;
  std::memset(&a, 0, sizeof a);
  for (int m = 0; m < n_moves; ++m) {
    if (static_cast<int64_t>(src_begin[m]) + n_tokens[m] > capacity ||
        static_cast<int64_t>(dst_begin[m]) + n_tokens[m] > capacity)
      return HW_ERR_CAPACITY;
    if (n_tokens[m] == 0 || src_begin[m] == dst_begin[m]) continue;  // nothing moves
    a.src[a.n_moves] = src_begin[m];
    a.dst[a.n_moves] = dst_begin[m];
    a.n[a.n_moves++] = n_tokens[m];
  }
  if (rows == 0 || a.n_moves == 0) return HW_OK;
  if (!k_cache || !v_cache || (dtype == HW_FP4_E2M1) != (kv_scale != nullptr)) return HW_ERR_INVALID;
  if (any_misaligned({k_cache, v_cache}, 16) || any_misaligned({kv_scale}, 4)) return HW_ERR_INVALID;
  const int64_t span = rows * capacity * row, scales = kv_scale ? rows * capacity * 4 : 0;
  if (spans_meet(k_cache, span, v_cache, span) || spans_meet(k_cache, span, kv_scale, scales) ||
      spans_meet(v_cache, span, kv_scale, scales))
    return HW_ERR_OVERLAP;
  for (int m = 0; m < a.n_moves; ++m) {
    for (int e = 0; e <= m; ++e) {
      const bool written = meets(a.dst[e], a.n[e], a.src[m], a.n[m]);  // e's destination is read by m
      const bool twice = e < m && meets(a.dst[e], a.n[e], a.dst[m], a.n[m]);
      const bool read = meets(a.src[e], a.n[e], a.dst[m], a.n[m]);  // e's source is overwritten by m
      if (written || twice || read) a.ordered = 1;
      if (e < m && (written || twice)) a.drain[m >> 5] |= 1u << (m & 31);
    }
  }
  a.pool[0] = static_cast<uint8_t *>(k_cache);
  a.pool[1] = static_cast<uint8_t *>(v_cache);
  a.kv_scale = static_cast<uint32_t *>(kv_scale);
  a.capacity = capacity;
  a.rows = static_cast<int32_t>(rows);
  a.row_bytes = row;
  const cudaError_t e = launch_move(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

int hw_block_move_status(int32_t *flags, void *stream) {
  if (!flags) return HW_ERR_INVALID;
  *flags = 0;
  const cudaError_t e = read_move_flags(flags, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

int hw_compact_moves(int32_t n_blocks, const int32_t *block_start, const int32_t *block_len, const int32_t *room,
                     int64_t capacity, int32_t *new_start, int32_t *n_moves, int32_t *src_begin,
                     int32_t *n_tokens, int32_t *dst_begin) {
  if (n_blocks < 0 || capacity < 0) return HW_ERR_INVALID;
  if (n_blocks > HW_MAX_MOVES || capacity > INT32_MAX) return HW_ERR_UNSUPPORTED;
  if (!n_moves || (n_blocks > 0 && (!block_start || !block_len || !new_start || !src_begin || !n_tokens || !dst_begin)))
    return HW_ERR_INVALID;
  int order_of[HW_MAX_MOVES];
  std::iota(order_of, order_of + n_blocks, 0);
  // (an empty block stands before one that starts at the same token)
  std::sort(order_of, order_of + n_blocks, [&](int x, int y) {
    if (block_start[x] != block_start[y]) return block_start[x] < block_start[y];
    return block_len[x] != block_len[y] ? block_len[x] < block_len[y] : x < y;
  });
  const struct {
    const int *b, *e;
    const int *begin() const { return b; }
    const int *end() const { return e; }
  } order = {order_of, order_of + n_blocks};
  int64_t end = 0, at = 0;
  for (const int b : order) {
    if (block_start[b] < 0 || block_len[b] < 0 || (room && room[b] < 0)) return HW_ERR_INVALID;
    if (static_cast<int64_t>(block_start[b]) + block_len[b] > capacity) return HW_ERR_CAPACITY;
    if (block_len[b] > 0 && block_start[b] < end) return HW_ERR_OVERLAP;
    end = std::max(end, static_cast<int64_t>(block_start[b]) + block_len[b]);
    at += static_cast<int64_t>(block_len[b]) + (room ? room[b] : 0);
    if (at > capacity) return HW_ERR_CAPACITY;
  }
  at = 0;
  for (const int b : order) {
    new_start[b] = static_cast<int32_t>(at);
    at += static_cast<int64_t>(block_len[b]) + (room ? room[b] : 0);
  }
  // down-moves from the lowest block on, then up-moves from the highest: no move
  // writes over tokens that a later one still has to read
  int n = 0;
  auto put = [&](int b) {
    src_begin[n] = block_start[b];
    n_tokens[n] = block_len[b];
    dst_begin[n++] = new_start[b];
  };
  for (const int b : order)
    if (block_len[b] > 0 && new_start[b] < block_start[b]) put(b);
  for (int i = n_blocks - 1; i >= 0; --i)
    if (block_len[order_of[i]] > 0 && new_start[order_of[i]] > block_start[order_of[i]]) put(order_of[i]);
  *n_moves = n;
  return HW_OK;
}

}  // extern "C"
