// tree_api.cpp - the draft-tree entry points of the C ABI (declared in
// include/hogwild.h): argument checks on the host, workspace layout, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "hogwild.h"
#include "hw_internal.h"
#include "hw_tree.h"

namespace hw {

// Description checks of the tree calls; OK also for empty descriptions.
static int check_tree(const hw_attn_desc *d, int32_t max_nodes) {
  const int st = check_desc(d);
  if (st != HW_OK) return st;
  if (max_nodes <= 0) return HW_ERR_INVALID;
  if (d->flags & HW_DESC_VIEW_LIMITS) return HW_ERR_UNSUPPORTED;
  if (max_nodes > HW_MAX_TREE_NODES || d->n_rows > HW_MAX_VIEW_ENTRIES) return HW_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->n_rows) * max_nodes > HW_MAX_TREE_QUERIES) return HW_ERR_UNSUPPORTED;
  return HW_OK;
}

// The workspace checked against the description, and the kernels' arguments.
static int tree_args(TreeArgs &a, const hw_attn_desc *d, int32_t max_nodes, void *workspace,
                     size_t workspace_bytes) {
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return HW_ERR_WORKSPACE;
  const int sms = device_sm_count();
  if (sms <= 0) return cuda_fail(cudaGetLastError());
  std::memset(&a, 0, sizeof a);
  a.L = tree_layout(*d, max_nodes, sms);
  if (workspace_bytes < a.L.total) return HW_ERR_WORKSPACE;
  a.ws = static_cast<uint8_t *>(workspace);
  a.n_rows = d->n_rows;
  a.max_nodes = max_nodes;
  a.n_q_heads = d->n_q_heads;
  a.n_kv_heads = d->n_kv_heads;
  a.head_dim = d->head_dim;
  a.n_blocks = d->n_blocks;
  a.n_view = d->max_view_blocks;
  a.dtype = d->dtype;
  a.capacity = d->cache_capacity;
  a.rope_theta = d->rope_theta;
  a.scale_log2 = static_cast<float>(static_cast<double>(d->scale) * 1.4426950408889634074);
  rope_phase_table(d->head_dim, d->rope_theta, a.phase);
  return HW_OK;
}

static bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

static int decode_tree(const hw_attn_desc *d, int32_t max_nodes, const void *q, const void *k_new,
                       const void *v_new, void *k_cache, void *v_cache, const float *k_scale,
                       const float *v_scale, void *out, float *lse, void *workspace,
                       size_t workspace_bytes, void *stream) {
  if (d->n_rows == 0) return HW_OK;
  if (!q || !k_new || !v_new || !out) return HW_ERR_INVALID;
  if (misaligned(q) || misaligned(k_new) || misaligned(v_new)) return HW_ERR_INVALID;
  const bool have_pool = d->n_blocks > 0 && d->cache_capacity > 0;
  if (have_pool && (!k_cache || !v_cache || misaligned(k_cache) || misaligned(v_cache)))
    return HW_ERR_INVALID;
  TreeArgs a;
  const int st = tree_args(a, d, max_nodes, workspace, workspace_bytes);
  if (st != HW_OK) return st;
  if (!have_pool) return HW_OK;  // no tree has a place: nothing to attend
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k = k_cache;
  a.v = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.out = out;
  a.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_tree_append(a, s);
  if (e == cudaSuccess && tree_on_tensor_cores(d->dtype, d->head_dim)) {
    CUtensorMap km, vm;
    const bool e4m3 = d->dtype == HW_FP8_E4M3;
    if (!make_pool_map(&km, k_cache, d->cache_capacity, d->n_kv_heads, e4m3) ||
        !make_pool_map(&vm, v_cache, d->cache_capacity, d->n_kv_heads, e4m3))
      return cuda_fail(cudaErrorInvalidValue);
    e = launch_tree_tc(a, km, vm, s);
  } else if (e == cudaSuccess) {
    e = launch_tree_simt(a, s);
  }
  if (e == cudaSuccess) e = launch_tree_merge(a, s);
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

}  // namespace hw

using namespace hw;

extern "C" {

int hw_attn_tree_workspace_size(const hw_attn_desc *d, int32_t max_nodes, size_t *bytes) {
  const int st = check_tree(d, max_nodes);
  if (st != HW_OK) return st;
  if (!bytes) return HW_ERR_INVALID;
  const int sms = device_sm_count();
  if (sms <= 0) return cuda_fail(cudaGetLastError());
  *bytes = tree_layout(*d, max_nodes, sms).total;
  return HW_OK;
}

int hw_attn_plan_tree(const hw_attn_desc *d, int32_t max_nodes, const int32_t *block_start,
                      const int32_t *block_len, const int32_t *view_block,
                      const int32_t *view_offset, const int32_t *q_pos, const int32_t *q_to_kv,
                      const int32_t *tree_block, const int32_t *tree_start, const int32_t *n_nodes,
                      const int32_t *parent, void *workspace, size_t workspace_bytes,
                      void *stream) {
  int st = check_tree(d, max_nodes);
  if (st != HW_OK) return st;
  if (d->n_rows == 0) return HW_OK;
  if (!q_pos || !tree_block || !n_nodes || !parent) return HW_ERR_INVALID;
  if (d->max_view_blocks > 0 && (!view_block || !view_offset)) return HW_ERR_INVALID;
  if (d->n_blocks > 0 && (!block_start || !block_len)) return HW_ERR_INVALID;
  TreeArgs a;
  st = tree_args(a, d, max_nodes, workspace, workspace_bytes);
  if (st != HW_OK) return st;
  const TreeMeta m = {block_start, block_len, view_block, view_offset, q_pos, q_to_kv,
                      tree_block, tree_start, n_nodes, parent};
  const cudaError_t e = launch_tree_plan(a, m, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

int hw_attn_decode_tree(const hw_attn_desc *d, int32_t max_nodes, const void *q, const void *k_new,
                        const void *v_new, void *k_cache, void *v_cache, void *out, float *lse,
                        void *workspace, size_t workspace_bytes, void *stream) {
  const int st = check_tree(d, max_nodes);
  if (st != HW_OK) return st;
  if (d->dtype == HW_FP8_E4M3) return HW_ERR_UNSUPPORTED;  // the _fp8 form takes the scales
  return decode_tree(d, max_nodes, q, k_new, v_new, k_cache, v_cache, nullptr, nullptr, out, lse,
                     workspace, workspace_bytes, stream);
}

int hw_attn_decode_tree_fp8(const hw_attn_desc *d, int32_t max_nodes, const void *q,
                            const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                            const float *k_scale, const float *v_scale, void *out, float *lse,
                            void *workspace, size_t workspace_bytes, void *stream) {
  const int st = check_tree(d, max_nodes);
  if (st != HW_OK) return st;
  if (d->dtype != HW_FP8_E4M3) return HW_ERR_INVALID;
  if (d->n_rows > 0 && (!k_scale || !v_scale)) return HW_ERR_INVALID;
  return decode_tree(d, max_nodes, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, out, lse,
                     workspace, workspace_bytes, stream);
}

int hw_tree_commit(const hw_attn_desc *d, int32_t max_nodes, int32_t n_layers, void *k_cache,
                   void *v_cache, const int32_t *path, const int32_t *n_path, void *workspace,
                   size_t workspace_bytes, void *stream) {
  int st = check_tree(d, max_nodes);
  if (st != HW_OK) return st;
  if (n_layers < 0) return HW_ERR_INVALID;
  if (d->n_rows == 0 || n_layers == 0) return HW_OK;
  if (!path || !n_path) return HW_ERR_INVALID;
  const bool have_pool = d->n_blocks > 0 && d->cache_capacity > 0;
  if (have_pool && (!k_cache || !v_cache || misaligned(k_cache) || misaligned(v_cache)))
    return HW_ERR_INVALID;
  TreeArgs a;
  st = tree_args(a, d, max_nodes, workspace, workspace_bytes);
  if (st != HW_OK) return st;
  if (!have_pool) return HW_OK;
  const int esz = d->dtype == HW_F32 ? 4 : d->dtype == HW_FP8_E4M3 ? 1 : 2;
  const TreeCommitArgs c = {k_cache, v_cache, path, n_path, n_layers, esz};
  const cudaError_t e = launch_tree_commit(a, c, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

int hw_tree_verify(int32_t dtype, int32_t n_rows, int32_t max_nodes, int32_t vocab,
                   const int32_t *n_nodes, const int32_t *parent, const int32_t *token,
                   const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                   const float *u_accept, const float *u_sample, int32_t *path, int32_t *n_path,
                   int32_t *next_token, void *stream) {
  if (dtype != HW_F32 && dtype != HW_BF16) return HW_ERR_INVALID;
  if (n_rows < 0 || max_nodes <= 0 || vocab <= 0) return HW_ERR_INVALID;
  if (p_stride < vocab || (q && q_stride < vocab)) return HW_ERR_INVALID;
  if (max_nodes > HW_MAX_TREE_NODES || vocab > HW_MAX_VOCAB) return HW_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(n_rows) * max_nodes > HW_MAX_TREE_QUERIES) return HW_ERR_UNSUPPORTED;
  if (n_rows == 0) return HW_OK;
  if (!n_nodes || !parent || !token || !p || !u_accept || !u_sample || !path || !n_path || !next_token)
    return HW_ERR_INVALID;
  const uintptr_t esz = dtype == HW_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & (esz - 1)) return HW_ERR_INVALID;
  const TreeVerifyArgs a = {p, q, p_stride, q_stride, n_nodes, parent, token, u_accept, u_sample,
                            path, n_path, next_token, n_rows, max_nodes, vocab, dtype, 0};
  const cudaError_t e = launch_tree_verify(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HW_OK : cuda_fail(e);
}

}  // extern "C"
