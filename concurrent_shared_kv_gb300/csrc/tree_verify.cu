// tree_verify.cu - drafted tokens held against the target's probabilities,
// from given random numbers, and the token that follows the accepted ones.
//
// At a node the children are tried in order.  After k rejections the
// target's distribution is the normalised remainder max(p'_k-1 - q, 0);
// written without the divisions it stays one expression,
//   a_k(x) = max(p(x) - c_k q(x), 0),  s_k = sum_x a_k(x),  c_0 = 0, s_0 = 1,
//   c_k+1 = c_k + s_k,  p'_k = a_k / s_k,
// (where a_k-1 is 0, p - c_k q is negative too).  Child x stands if
// u q(x) s_k < a_k(x); with none left, the next token is the first x whose
// running sum of a_k passes u s.
//
// Arithmetic: unsigned fixed point, 56 bits behind the point.  A probability
// from 2^-32 up is exact, smaller ones and the products lose less than 2^-56
// each, and sums do not depend on their order, so the decisions are those of
// a 64-bit evaluation and the same on every run.  (fp32 sums would misplace
// the drawn token with a probability of about vocab x 2^-27.)
//
// One cluster of 8 CTAs a row: the vocabulary is cut into one slice a warp,
// a rejection costs one pass over the node's two rows of probabilities, and
// the slices' sums are joined through distributed shared memory.  Everything
// else needs single values: every drafted token's p and q are fetched at
// once, so a path of any depth waits for memory once.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "hw_tree.h"

namespace hw {

namespace {

namespace cg = cooperative_groups;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kSlices = kCluster * kWarps;
constexpr int kShift = 56;
constexpr uint64_t kOne = 1ull << kShift;

// x in fixed point: NaN and negative values count as 0, values over 1 as 1.
__device__ __forceinline__ uint64_t to_fix(float x) {
  return x > 0.f ? (x < 1.f ? __float2ull_rz(x * 0x1p56f) : kOne) : 0;
}
// floor(a b) of two fixed-point numbers, the product below 2^8.
__device__ __forceinline__ uint64_t mul_fix(uint64_t a, uint64_t b) {
  return (__umul64hi(a, b) << (64 - kShift)) | ((a * b) >> kShift);
}
__device__ __forceinline__ uint64_t left_of(uint64_t p, uint64_t c, uint64_t q) {
  const uint64_t t = mul_fix(c, q);
  return p > t ? p - t : 0;
}

// A row of probabilities.  Vector loads start at multiples of four elements
// of memory, so positions count from the last such multiple at or before the
// row: y = x + off.
template <typename T>
struct Row {
  const T *at;  // position 0
  int off, end;  // first position, one past the last
  __device__ __forceinline__ Row(const T *row, int vocab) {
    off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 3);
    at = row - off;
    end = off + vocab;
  }
};
__device__ __forceinline__ float one(const float *p) { return *p; }
__device__ __forceinline__ float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void four(const float *p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void four(const __nv_bfloat16 *p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}
// Positions y .. y+3 of p (y a multiple of 4), 0 outside the row.
template <typename T>
__device__ __forceinline__ void load_p(const Row<T> &r, int y, float (&x)[4]) {
  if (y >= r.off && y + 4 <= r.end) {
    four(r.at + y, x);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = y + e >= r.off && y + e < r.end ? one(r.at + y + e) : 0.f;
  }
}
// The same tokens of q, whose row may lie otherwise in memory.
template <typename T>
__device__ __forceinline__ void load_q(const Row<T> &p, const Row<T> &q, int y, float (&x)[4]) {
  if (p.off == q.off) {
    load_p(q, y, x);
  } else {
    const int d = q.off - p.off;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = y + e >= p.off && y + e < p.end ? one(q.at + y + e + d) : 0.f;
  }
}

struct Smem {
  int32_t parent[kMaxNodes], token[kMaxNodes];
  uint64_t px[kMaxNodes], qx[kMaxNodes], u[kMaxNodes];
  uint64_t wsum[kWarps];
  uint64_t total[2][kCluster];  // per pass parity: every CTA's sum
  uint64_t scan[kWarps];
  int32_t path[kMaxNodes], gone[kMaxNodes];  // accepted nodes; tokens removed at the current node
  // the walk, written by thread 0
  int32_t cur, next, n_path, n_gone, again;
  uint64_t c, s;
  int32_t bad;
  int32_t slice;   // the drawn token's warp slice in this CTA, or -1
  uint64_t target;  // what is left of the draw there
};

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    tree_verify_kernel(const __grid_constant__ TreeVerifyArgs a) {
  __shared__ Smem S;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int r = blockIdx.x / kCluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TN = a.max_nodes, V = a.vocab, n = a.n_nodes[r];
  const T *p0 = static_cast<const T *>(a.p) + static_cast<int64_t>(r) * TN * a.p_stride;
  const T *q0 = a.q ? static_cast<const T *>(a.q) + static_cast<int64_t>(r) * TN * a.q_stride : nullptr;
  if (tid == 0) S.bad = n < 0 || n > TN;
  __syncthreads();
  if (!S.bad && tid < n) {
    const int64_t at = static_cast<int64_t>(r) * TN + tid;
    const int par = a.parent[at], tok = a.token[at];
    S.parent[tid] = par;
    S.token[tid] = tok;
    const bool root = tid == 0;
    if (par < -1 || par >= tid || (!root && (tok < 0 || tok >= V))) {
      S.bad = 1;
    } else if (par >= 0) {
      S.px[tid] = to_fix(one(p0 + par * a.p_stride + tok));
      S.qx[tid] = q0 ? to_fix(one(q0 + par * a.q_stride + tok)) : kOne;
      S.u[tid] = to_fix(a.u_accept[at]);
    }
  }
  __syncthreads();
  if (S.bad || n == 0) {  // (the same in every CTA of the cluster)
    if (rank == 0) {
      for (int j = tid; j < TN; j += kThreads) a.path[static_cast<int64_t>(r) * TN + j] = -1;
      if (tid == 0) {
        a.n_path[r] = 0;
        a.next_token[r] = -1;
      }
    }
    return;
  }
  if (tid == 0) {
    S.cur = 0;
    S.next = 1;
    S.path[0] = 0;
    S.n_path = 1;
    S.n_gone = 0;
    S.c = 0;
    S.s = kOne;
  }
  // positions of a warp's slice: whole groups of 128 (a lane's 4 x 32 lanes)
  const int per = ((V + 3 + kSlices - 1) / kSlices + 127) / 128 * 128;
  int parity = 0;
  uint64_t c_pass = 0, c_kept = 0;
  bool fresh = false;  // the slices' sums are those of (cur, c)
  for (;;) {
    if (tid == 0) {
      // on to the next rejection that needs a sum, or to the end
      int cur = S.cur, i = S.next, again = 0;
      bool moved = false;
      for (; i < n && !again; ++i) {
        if (S.parent[i] != cur) continue;
        uint64_t rest = left_of(S.px[i], S.c, S.qx[i]);
        if (!q0) {
          rest = S.px[i];
          for (int j = 0; j < S.n_gone; ++j)
            if (S.gone[j] == S.token[i]) rest = 0;
        }
        if (mul_fix(mul_fix(S.u[i], S.qx[i]), S.s) < rest) {
          cur = i;
          S.path[S.n_path++] = i;
          S.n_gone = 0;
          S.c = 0;
          S.s = kOne;
          moved = true;
        } else if (!q0) {
          if (rest > 0) S.gone[S.n_gone++] = S.token[i];
          S.s = S.s > rest ? S.s - rest : 0;
          moved = true;
        } else {
          again = 1;
        }
      }
      S.cur = cur;
      S.next = i;
      S.again = again | (moved ? 2 : 0);
    }
    __syncthreads();
    const int again = S.again;
    if (again & 2) fresh = false;
    c_kept = S.c;
    if (!(again & 1) && fresh) break;
    // one pass: the slices' sums of max(p - c q, 0)
    c_pass = again & 1 ? c_kept + S.s : c_kept;
    const Row<T> p(p0 + S.cur * a.p_stride, V);
    uint64_t sum = 0;
    const int y0 = (rank * kWarps + warp) * per, y1 = min(y0 + per, p.end);
    if (c_pass == 0) {
#pragma unroll 4
      for (int y = y0 + 4 * lane; y < y1; y += 128) {
        float x[4];
        load_p(p, y, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += to_fix(x[e]);
      }
    } else {
      const Row<T> q(q0 + S.cur * a.q_stride, V);
#pragma unroll 4
      for (int y = y0 + 4 * lane; y < y1; y += 128) {
        float x[4], z[4];
        load_p(p, y, x);
        load_q(p, q, y, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += left_of(to_fix(x[e]), c_pass, to_fix(z[e]));
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) S.wsum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      for (int j = 0; j < S.n_gone; ++j) {  // tokens removed at this node
        const int y = S.gone[j] + p.off, w = y / per - rank * kWarps;
        if (w >= 0 && w < kWarps) S.wsum[w] -= to_fix(one(p.at + y));
      }
      uint64_t t = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += S.wsum[w];
      S.scan[0] = t;
    }
    __syncthreads();
    if (tid < kCluster) cluster.map_shared_rank(&S, tid)->total[parity][rank] = S.scan[0];
    cluster.sync();
    if (again & 1) {
      uint64_t t = 0;
#pragma unroll
      for (int x = 0; x < kCluster; ++x) t += S.total[parity][x];
      fresh = t > 0;  // nothing left: the distribution before the rejection stays
      __syncthreads();
      if (tid == 0 && t > 0) {
        S.c = c_pass;
        S.s = t;
      }
    } else {
      fresh = true;
    }
    parity ^= 1;
    __syncthreads();
  }
  parity ^= 1;  // the last pass's
  // the draw: this CTA's and its warps' share of the running sum
  if (tid == 0) {
    uint64_t all = 0, before = 0;
    for (int x = 0; x < kCluster; ++x) {
      if (x == rank) before = all;
      all += S.total[parity][x];
    }
    S.slice = -1;
    if (all > 0) {
      uint64_t t = mul_fix(to_fix(a.u_sample[r]), all);
      if (t >= all) t = all - 1;
      if (t >= before && t - before < S.total[parity][rank]) {
        t -= before;
        int w = 0;
        while (t >= S.wsum[w]) t -= S.wsum[w++];
        S.slice = w;
        S.target = t;
      }
    } else if (rank == 0) {
      a.next_token[r] = -1;
    }
  }
  if (rank == 0) {
    const int np = S.n_path;
    for (int j = tid; j < TN; j += kThreads) a.path[static_cast<int64_t>(r) * TN + j] = j < np ? S.path[j] : -1;
    if (tid == 0) a.n_path[r] = np;
  }
  __syncthreads();
  if (S.slice < 0) return;
  // the owner goes over the slice once more, four positions a thread
  const Row<T> p(p0 + S.cur * a.p_stride, V);
  const int y0 = (rank * kWarps + S.slice) * per, y1 = min(y0 + per, p.end);
  const uint64_t c = S.c;
  uint64_t target = S.target;
  for (int yb = y0; yb < y1; yb += 4 * kThreads) {
    const int y = yb + 4 * tid;
    uint64_t v[4] = {0, 0, 0, 0}, mine = 0;
    if (y < y1) {
      float x[4];
      load_p(p, y, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = to_fix(x[e]);
      if (c != 0) {
        const Row<T> q(q0 + S.cur * a.q_stride, V);
        float z[4];
        load_q(p, q, y, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = left_of(v[e], c, to_fix(z[e]));
      }
      for (int j = 0; j < S.n_gone; ++j) {
        const int e = S.gone[j] + p.off - y;
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2)
          if (e == e2) v[e2] = 0;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) mine += v[e];
    }
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) S.scan[warp] = incl;
    __syncthreads();
    uint64_t before = incl - mine, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += S.scan[w];
      all += S.scan[w];
    }
    if (target >= before && target - before < mine) {
      uint64_t t = target - before;
      int e = 0;
      while (t >= v[e]) t -= v[e++];
      a.next_token[r] = y + e - p.off;
    }
    if (target < all) break;  // (the same in every thread)
    target -= all;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_tree_verify(const TreeVerifyArgs &a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.n_rows) * kCluster;
  if (a.dtype == HW_F32)
    tree_verify_kernel<float><<<grid, kThreads, 0, s>>>(a);
  else
    tree_verify_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace hw
