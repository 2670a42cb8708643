// tree_simt.cu - attention for trees of drafted tokens on the CUDA cores
// (fp32 FMA, fp32 accumulation): fp32 caches, where tensor-core rounding is
// too coarse, and head_dim 64.
//
// A CTA walks its units (hw_tree.h): per group up to 32 queries in shared
// memory, rotated anew for every span, tiles of 64 tokens, an online softmax
// in the log2 domain, and a record of (m, l, o) per column at the end.  A
// tree's tile is masked with the ancestor bits of each column's node.
// Bound by shared memory: 12 wavefronts of loads for 8 clocks of FMAs in the
// scores (a warp's 4 queries share a key's load; a query at a time it was 36),
// 20 for 16 in P.V, and by tiles loaded without anything under way beside them
// but the SM's other CTAs.  4 trees of 16 nodes over 16K tokens (40/8 heads):
// bf16 with head_dim 64 0.51 ms, fp32 with 128 1.26 ms, 18 TFLOP/s; 2 trees of
// 6 nodes over 256 fp32 tokens (4/2 heads) 13.5 us, all latency.
#include "hw_device.cuh"
#include "hw_tree.h"

namespace hw {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr int kCols = 32;
constexpr int kPerWarp = kCols / (kThreads / 32);  // queries of a warp

template <int D>
struct Smem {
  alignas(16) float q[kCols][D + 4];
  alignas(16) float k[kTile][D + 4];
  alignas(16) float v[kTile][D + 4];
  alignas(16) float p[kCols][kTile + 4];
  float m[kCols], l[kCols], alpha[kCols];
  TreeColumn col[kCols];
  int32_t rot[kCols];     // row of the rotation table for this span, or -1: unseen
  uint32_t bad[2];        // a partial tile's tokens with a value that is not finite
};

// The scores of N queries (warp, warp + 8, ..) against tokens lane and
// lane + 32, before scaling.  A key's four elements are loaded once for all N.
template <int D, int N>
__device__ __forceinline__ void scores(const Smem<D> &S, int warp, int lane, float (&s)[kPerWarp][2]) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i][0] = s[i][1] = 0.f;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    const float4 k0 = *reinterpret_cast<const float4 *>(&S.k[lane][d]);
    const float4 k1 = *reinterpret_cast<const float4 *>(&S.k[lane + 32][d]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 q = *reinterpret_cast<const float4 *>(&S.q[warp + i * (kThreads / 32)][d]);
      s[i][0] += q.x * k0.x + q.y * k0.y + q.z * k0.z + q.w * k0.w;
      s[i][1] += q.x * k1.x + q.y * k1.y + q.z * k1.z + q.w * k1.w;
    }
  }
}

template <typename T>
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
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D> &S = *reinterpret_cast<Smem<D> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = blockIdx.x;
  TreeCta at = tree_at<TreeCta>(a, a.L.ctas)[c];
  const TreeHeader &hdr = *tree_at<const TreeHeader>(a, a.L.hdr);
  const bool ok = tree_plan_ok(a), work = ok && c < hdr.n_ctas;
  if (!ok && tid == 0) flag_error(reinterpret_cast<int32_t *>(a.ws), HW_DEV_BAD_PLAN);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the trees' tokens
  if (!work) return;
  const TreeGroup *groups = tree_at<TreeGroup>(a, a.L.groups);
  const TreeSpan *spans = tree_at<TreeSpan>(a, a.L.spans);
  const int G = a.n_q_heads / a.n_kv_heads;
  constexpr int EPV = 16 / sizeof(T), CPR = D / EPV;
  constexpr int QSTEP = kThreads / D;   // columns side by side in P.V
  constexpr int QPT = kCols / QSTEP;    // columns of a thread
  const int dcol = tid % D, qfirst = tid / D;

  while (at.n_units > 0) {
    const TreeGroup gr = groups[at.group];
    const int h = at.head, nq = gr.n_cols;
    if (tid < nq) {
      S.col[tid] = tree_at<TreeColumn>(a, a.L.columns)[gr.col0 + tid];
      S.m[tid] = kNoScore;
      S.l[tid] = 0.f;
    }
    float acc[QPT];
#pragma unroll
    for (int k = 0; k < QPT; ++k) acc[k] = 0.f;
    for (; at.span < gr.n_spans && at.n_units > 0; ++at.span, at.tile = 0) {
      const TreeSpan sp = spans[gr.span0 + at.span];
      __syncthreads();
      if (tid < nq) {  // the columns that see the span, and their rotations
        const TreeColumn &cl = S.col[tid];
        const int v = sp.row < 0 ? tree_at<int16_t>(a, a.L.map)[sp.map + cl.row] : cl.node / a.max_nodes == sp.row ? a.n_view : -1;
        S.rot[tid] = v < 0 ? -1 : cl.rot + v * cl.n_nodes;
      }
      __syncthreads();
      for (int x = tid; x < nq * (D / 2); x += kThreads) {
        const int qi = x / (D / 2), i = x % (D / 2);
        if (S.rot[qi] < 0) continue;
        const int64_t row = static_cast<int64_t>(S.col[qi].node) * a.n_q_heads + tree_at<int32_t>(a, a.L.heads)[h * G + S.col[qi].head];
        const T *qp = reinterpret_cast<const T *>(a.q) + row * D;
        const float x0 = to_f32<T>(qp[i]), x1 = to_f32<T>(qp[i + D / 2]);
        const float2 r = tree_at<float2>(a, a.L.rot)[static_cast<int64_t>(S.rot[qi]) * (D / 2) + i];
        S.q[qi][i] = x0 * r.x - x1 * r.y;
        S.q[qi][i + D / 2] = x1 * r.x + x0 * r.y;
      }
      const int t1 = min((sp.len + kTile - 1) / kTile, at.tile + at.n_units);
      at.n_units -= t1 - at.tile;
      for (int t = at.tile; t < t1; ++t) {
        const int valid = min(kTile, sp.len - t * kTile);
        const int64_t row0 = static_cast<int64_t>(h) * a.capacity + sp.start + t * kTile;
        const T *kb = reinterpret_cast<const T *>(a.k) + row0 * D;
        const T *vb = reinterpret_cast<const T *>(a.v) + row0 * D;
        __syncthreads();
        if (tid < 2) S.bad[tid] = 0;
        __syncthreads();
        for (int x = tid; x < kTile * CPR; x += kThreads) {
          const int row = x / CPR, col = (x % CPR) * EPV;
          float kf[EPV], vf[EPV];
          if (row < valid) {
            unpack<T>(*reinterpret_cast<const uint4 *>(kb + static_cast<int64_t>(row) * D + col), kf);
            unpack<T>(*reinterpret_cast<const uint4 *>(vb + static_cast<int64_t>(row) * D + col), vf);
          } else {  // rows past the span may hold anything
#pragma unroll
            for (int i = 0; i < EPV; ++i) kf[i] = vf[i] = 0.f;
          }
          if (sp.partial) {
            // 0 * NaN must not reach the columns that do not see the token;
            // those that do get a NaN through their sum
#pragma unroll
            for (int i = 0; i < EPV; ++i)
              if (!(fabsf(vf[i]) < INFINITY)) {
                vf[i] = 0.f;
                atomicOr(&S.bad[row >> 5], 1u << (row & 31));
              }
          }
#pragma unroll
          for (int i = 0; i < EPV; i += 4) {
            *reinterpret_cast<float4 *>(&S.k[row][col + i]) = make_float4(kf[i], kf[i + 1], kf[i + 2], kf[i + 3]);
            *reinterpret_cast<float4 *>(&S.v[row][col + i]) = make_float4(vf[i], vf[i + 1], vf[i + 2], vf[i + 3]);
          }
        }
        __syncthreads();
        float score[kPerWarp][2];
        switch ((nq - warp + kThreads / 32 - 1) / (kThreads / 32)) {  // this warp's queries
          case 4: scores<D, 4>(S, warp, lane, score); break;
          case 3: scores<D, 3>(S, warp, lane, score); break;
          case 2: scores<D, 2>(S, warp, lane, score); break;
          default: scores<D, 1>(S, warp, lane, score); break;
        }
#pragma unroll
        for (int i = 0; i < kPerWarp; ++i) {
          const int qq = warp + i * (kThreads / 32);
          if (qq >= nq) break;
          float s0 = score[i][0], s1 = score[i][1];
          const bool seen = S.rot[qq] >= 0;
          bool in0 = seen && lane < valid, in1 = seen && lane + 32 < valid;
          if (sp.row >= 0) {  // a tree: the node's ancestors and itself
            const uint32_t *mask = tree_at<uint32_t>(a, a.L.mask) + static_cast<int64_t>(S.col[qq].node) * 4 + 2 * t;
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
          const float p0 = ex2(s0 - m_new), p1 = ex2(s1 - m_new);
          float sum = p0 + p1;
          if ((in0 && (S.bad[0] >> lane) & 1u) || (in1 && (S.bad[1] >> lane) & 1u)) sum = NAN;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          S.p[qq][lane] = p0;
          S.p[qq][lane + 32] = p1;
          if (lane == 0) {
            const float alpha = ex2(m_old - m_new);
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
    }
    // the record
    const int64_t k = static_cast<int64_t>(h) * hdr.n_groups + at.group;
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
    at.span = at.tile = 0;
    if (++at.group == hdr.n_groups) {  // (no group is wide here)
      at.group = 0;
      ++at.head;
    }
  }
}

template <typename T, int D>
cudaError_t launch(const TreeArgs &a, cudaStream_t s) {
  const size_t smem = sizeof(Smem<D>);
  static bool configured = false;
  if (!configured) {
    const cudaError_t e = cudaFuncSetAttribute(tree_simt_kernel<T, D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    configured = true;
  }
  // a dependent of the append launch (tree_plan.cu), started while that ends
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.L.ctas_max);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_simt_kernel<T, D>, a);
}

}  // namespace

cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t s) {
  if (a.dtype == HW_BF16) return launch<__nv_bfloat16, 64>(a, s);
  return a.head_dim == 64 ? launch<float, 64>(a, s) : launch<float, 128>(a, s);
}

}  // namespace hw
