// hw_cache.h - what cache_api.cpp hands to the kernels of cache_ops.cu and block_move.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hw_internal.h"

namespace hw {

// Tokens into (hw_cache_write) or out of (hw_cache_read) the pools.
struct CacheArgs {
  void *k_cache, *v_cache;   // [layers][Hkv][capacity][row]
  void *kv_scale;            // E2M1: [layers][Hkv][capacity] words (hw_fp4.cuh)
  const float *k_scale, *v_scale;  // E4M3: [layers][Hkv]
  const void *k_new, *v_new;  // write: [layers][n][Hkv][D]
  void *k_out, *v_out;        // read: likewise
  const int32_t *slot, *pos;
  int32_t *flags;  // HW_DEV_* bits, or null
  int32_t n_tokens, n_layers, n_kv_heads, head_dim;
  int64_t capacity;
  uint64_t phase[64];
};
cudaError_t launch_cache_write(const CacheArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_cache_read(const CacheArgs &a, int dtype, cudaStream_t s);

// hw_block_commit_many_fp4: commit_impl's arguments and the scales.
struct CommitScales {
  const uint32_t *src;
  uint32_t *dst;
};
cudaError_t launch_commit_fp4(const CommitArgs &a, const CommitScales &scales, cudaStream_t s);

// Token ranges moved within the pools, one after the other.
constexpr int kMaxMoves = HW_MAX_MOVES;
struct MoveArgs {
  uint8_t *pool[2];    // K, V: [rows][capacity][row_bytes], rows = layers * Hkv
  uint32_t *kv_scale;  // E2M1, else null: [rows][capacity]
  int64_t capacity;
  int32_t rows, row_bytes, n_moves;
  int32_t ordered;     // some move touches what another, or itself, reads or writes
  int32_t src[kMaxMoves], dst[kMaxMoves], n[kMaxMoves];
  uint32_t drain[kMaxMoves / 32];  // bit m: move m starts once the ones before it are written
};
cudaError_t launch_move(const MoveArgs &a, cudaStream_t s);
// The current device's HW_DEV_* bits of moves, read and cleared once `s` is done.
cudaError_t read_move_flags(int32_t *flags, cudaStream_t s);

}  // namespace hw
