// tree_simt.cu - attention for trees of drafted tokens on the CUDA cores
// (fp32 FMA, fp32 accumulation): fp32 caches, where tensor-core rounding is
// too coarse, and head_dim 64.
//
// A CTA walks its units (hw_tree.h): per segment up to 32 rotated queries in
// shared memory, tiles of 64 tokens, an online softmax in the log2 domain,
// and a record of (m, l, o) per column at the end.  A tree's tile is masked
// with the ancestor bits of each column's node.
#include <cuda_fp8.h>

#include "hw_device.cuh"
#include "hw_tree.h"

namespace hw {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr int kCols = 32;

template <int D>
struct Smem {
  alignas(16) float q[kCols][D + 4];
  alignas(16) float k[kTile][D + 4];
  alignas(16) float v[kTile][D + 4];
  alignas(16) float p[kCols][kTile + 4];
  float m[kCols], l[kCols], alpha[kCols];
  int32_t qrow[kCols];    // query row of the column: node * Hq + q head
  int32_t node[kCols];    // row * max_nodes + node
  int32_t rot[kCols];     // its row of the rotation table
};

template <typename KV>
__device__ __forceinline__ void unpack(const uint4 &u, float *x);
template <>
__device__ __forceinline__ void unpack<float>(const uint4 &u, float *x) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4 &u, float *x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void unpack<uint8_t>(const uint4 &u, float *x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> (16 * p)), __NV_E4M3));
      const float2 f = __half22float2(h);
      x[4 * i + 2 * p] = f.x;
      x[4 * i + 2 * p + 1] = f.y;
    }
}

// T: queries and outputs; KV: the cache's element (uint8_t: E4M3 codes).
template <typename T, typename KV, int D>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D> &S = *reinterpret_cast<Smem<D> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!tree_plan_ok(a)) {
    if (tid == 0) flag_error(reinterpret_cast<int32_t *>(a.ws), HW_DEV_BAD_PLAN);
    return;
  }
  const TreeHeader &hdr = *tree_at<const TreeHeader>(a, a.L.hdr);
  const int c = blockIdx.x;
  if (c >= hdr.n_ctas) return;
  TreeCta at = tree_at<TreeCta>(a, a.L.ctas)[c];
  const TreeSeg *segs = tree_at<TreeSeg>(a, a.L.segs);
  const TreeColumn *columns = tree_at<TreeColumn>(a, a.L.columns);
  const int G = a.n_q_heads / a.n_kv_heads;
  constexpr int EPV = 16 / sizeof(KV), CPR = D / EPV;
  constexpr int QSTEP = kThreads / D;   // columns side by side in P.V
  constexpr int QPT = kCols / QSTEP;    // columns of a thread
  const int dcol = tid % D, qfirst = tid / D;

  while (at.n_units > 0) {
    const TreeSeg sg = segs[at.seg];
    const int h = at.head, nq = sg.n_cols;
    const float ks = a.k_scale ? a.k_scale[h] : 1.f, vs = a.v_scale ? a.v_scale[h] : 1.f;
    if (tid < nq) {
      const TreeColumn tc = columns[sg.table + tid];
      S.node[tid] = tc.node;
      S.qrow[tid] = tc.node * a.n_q_heads + tree_at<int32_t>(a, a.L.heads)[h * G + tc.head];
      S.rot[tid] = tc.rot;
      S.m[tid] = -INFINITY;
      S.l[tid] = 0.f;
    }
    __syncthreads();
    for (int x = tid; x < nq * (D / 2); x += kThreads) {
      const int qi = x / (D / 2), i = x % (D / 2);
      const T *qp = reinterpret_cast<const T *>(a.q) + static_cast<int64_t>(S.qrow[qi]) * D;
      const float x0 = to_f32<T>(qp[i]), x1 = to_f32<T>(qp[i + D / 2]);
      const float2 r = tree_at<float2>(a, a.L.rot)[static_cast<int64_t>(S.rot[qi]) * (D / 2) + i];
      S.q[qi][i] = x0 * r.x - x1 * r.y;
      S.q[qi][i + D / 2] = x1 * r.x + x0 * r.y;
    }
    float acc[QPT];
#pragma unroll
    for (int k = 0; k < QPT; ++k) acc[k] = 0.f;
    const int tiles = (sg.len + kTile - 1) / kTile;
    const int t1 = min(tiles, at.tile + at.n_units);
    for (int t = at.tile; t < t1; ++t) {
      const int valid = min(kTile, sg.len - t * kTile);
      const int64_t row0 = static_cast<int64_t>(h) * a.capacity + sg.start + t * kTile;
      const KV *kb = reinterpret_cast<const KV *>(a.k) + row0 * D;
      const KV *vb = reinterpret_cast<const KV *>(a.v) + row0 * D;
      __syncthreads();
      for (int x = tid; x < kTile * CPR; x += kThreads) {
        const int row = x / CPR, col = (x % CPR) * EPV;
        float kf[EPV], vf[EPV];
        if (row < valid) {
          unpack<KV>(*reinterpret_cast<const uint4 *>(kb + static_cast<int64_t>(row) * D + col), kf);
          unpack<KV>(*reinterpret_cast<const uint4 *>(vb + static_cast<int64_t>(row) * D + col), vf);
        } else {  // rows past the segment may hold anything
#pragma unroll
          for (int i = 0; i < EPV; ++i) kf[i] = vf[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < EPV; ++i) {
          S.k[row][col + i] = kf[i] * ks;
          S.v[row][col + i] = vf[i] * vs;
        }
      }
      __syncthreads();
      for (int qq = warp; qq < nq; qq += kThreads / 32) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll 8
        for (int d = 0; d < D; d += 4) {
          const float4 qv = *reinterpret_cast<const float4 *>(&S.q[qq][d]);
          const float4 k0 = *reinterpret_cast<const float4 *>(&S.k[lane][d]);
          const float4 k1 = *reinterpret_cast<const float4 *>(&S.k[lane + 32][d]);
          s0 += qv.x * k0.x + qv.y * k0.y + qv.z * k0.z + qv.w * k0.w;
          s1 += qv.x * k1.x + qv.y * k1.y + qv.z * k1.z + qv.w * k1.w;
        }
        bool in0 = lane < valid, in1 = lane + 32 < valid;
        if (sg.row >= 0) {  // a tree: the node's ancestors and itself
          const uint32_t *mask = tree_at<uint32_t>(a, a.L.mask) + static_cast<int64_t>(S.node[qq]) * 4 + 2 * t;
          in0 = in0 && (mask[0] >> lane) & 1u;
          in1 = in1 && (mask[1] >> lane) & 1u;
        }
        s0 = in0 ? s0 * a.scale_log2 : -INFINITY;
        s1 = in1 ? s1 * a.scale_log2 : -INFINITY;
        float mx = fmaxf(s0, s1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_old = S.m[qq];
        const float m_new = fmaxf(m_old, mx);
        const float base = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: weights 0, no NaN
        const float p0 = ex2(s0 - base), p1 = ex2(s1 - base);
        float sum = p0 + p1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        S.p[qq][lane] = p0;
        S.p[qq][lane + 32] = p1;
        if (lane == 0) {
          const float alpha = ex2(m_old - base);
          S.alpha[qq] = alpha;
          S.m[qq] = m_new;
          S.l[qq] = S.l[qq] * alpha + sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < QPT; ++k) {
        const int qi = qfirst + k * QSTEP;
        if (qi < nq) acc[k] *= S.alpha[qi];
      }
      for (int tt = 0; tt < valid; tt += 4) {
        const float v0 = S.v[tt][dcol], v1 = S.v[tt + 1][dcol];
        const float v2 = S.v[tt + 2][dcol], v3 = S.v[tt + 3][dcol];
#pragma unroll
        for (int k = 0; k < QPT; ++k) {
          const int qi = qfirst + k * QSTEP;
          if (qi < nq) {
            const float4 pp = *reinterpret_cast<const float4 *>(&S.p[qi][tt]);
            acc[k] += pp.x * v0 + pp.y * v1 + pp.z * v2 + pp.w * v3;
          }
        }
      }
    }
    // the record
    const int64_t k = static_cast<int64_t>(h) * hdr.n_segs + at.seg;
    const int64_t rec = tree_at<int32_t>(a, a.L.piece_row)[k] +
                        static_cast<int64_t>(c - tree_at<int2>(a, a.L.piece_cta)[k].x) * nq;
#pragma unroll
    for (int k2 = 0; k2 < QPT; ++k2) {
      const int qi = qfirst + k2 * QSTEP;
      if (qi < nq) {
        tree_at<float>(a, a.L.o)[record_at(rec, nq, qi, dcol, D)] = acc[k2];
        if (dcol == 0) tree_at<float2>(a, a.L.ml)[rec + qi] = make_float2(S.m[qi], S.l[qi]);
      }
    }
    __syncthreads();
    at.n_units -= t1 - at.tile;
    at.tile = 0;
    if (++at.seg == hdr.n_segs) {
      at.seg = 0;
      ++at.head;
    }
  }
}

template <typename T, typename KV, int D>
cudaError_t launch(const TreeArgs &a, cudaStream_t s) {
  const size_t smem = sizeof(Smem<D>);
  static bool configured = false;
  if (!configured) {
    const cudaError_t e = cudaFuncSetAttribute(tree_simt_kernel<T, KV, D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    configured = true;
  }
  tree_simt_kernel<T, KV, D><<<a.L.ctas_max, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t s) {
  if (a.dtype == HW_FP8_E4M3) return launch<__nv_bfloat16, uint8_t, 128>(a, s);
  if (a.dtype == HW_BF16)
    return a.head_dim == 64 ? launch<__nv_bfloat16, __nv_bfloat16, 64>(a, s)
                            : launch<__nv_bfloat16, __nv_bfloat16, 128>(a, s);
  return a.head_dim == 64 ? launch<float, float, 64>(a, s) : launch<float, float, 128>(a, s);
}

}  // namespace hw
