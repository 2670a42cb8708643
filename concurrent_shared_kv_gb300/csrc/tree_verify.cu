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
// Arithmetic: what is decided is decided in integers, with 56 bits behind the
// point.  The single values of a test are exact (a probability from 2^-32 up)
// or lose less than 2^-56; an element of a sum is p - c q in fp32 with c as two
// floats - an error of 2^-24 of the difference itself - rounded to 56 bits
// behind the point and added as an integer.  Sums so do not depend on their
// order, runs repeat, and a running sum is off by some 2^-24 of its largest
// elements, where fp32 sums would misplace the drawn token once in a thousand
// draws.
//
// One cluster of 8 or 16 CTAs a row: the vocabulary is cut into one slice a warp,
// a rejection costs one pass over the node's two rows of probabilities, and
// the slices' sums are joined through distributed shared memory.  Everything
// else needs single values: every drafted token's p and q are fetched at
// once, so a path of any depth waits for memory once.
// Bound by latency: a launch, a cluster barrier a rejection, two trips to
// memory.  4 rows of 16 nodes over 131072 fp32 values 11.6 to 13.8 us, by the
// rejections there are (0.6 us of bytes), 64 rows of 8 nodes in bf16 24.6 to
// 26.3 us (5 us: two waves of clusters), 64 chosen nodes over 50021 values 9.5 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "hw_internal.h"
#include "hw_tree.h"

namespace hw {

namespace {

namespace cg = cooperative_groups;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
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
// c, with the same 56 bits behind the point: it grows by a row's sum, up to 128,
// with each of up to 127 rejections, to 2^14.
using Wide = unsigned __int128;
__device__ __forceinline__ uint64_t left_of(uint64_t p, Wide c, uint64_t q) {
  const Wide t = (c * q) >> kShift;  // (below 2^126)
  return p > t ? p - static_cast<uint64_t>(t) : 0;
}
// Packed fp32: two numbers an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// max(p - c q, 0) of two pairs held to [0, 1] (NaN counts as 0), c = c0 + c1.
template <bool kFirst>
__device__ __forceinline__ void left2(float &p0, float &p1, float c0, float c1, float q0, float q1) {
  const uint64_t p = pack2(__saturatef(p0), __saturatef(p1)), q = pack2(__saturatef(q0), __saturatef(q1));
  unpack2(kFirst ? fma2(pack2(-1.f, -1.f), q, p) : fma2(pack2(-c1, -c1), q, fma2(pack2(-c0, -c0), q, p)), p0, p1);
  p0 = fmaxf(p0, 0.f);
  p1 = fmaxf(p1, 0.f);
}
// Numbers in [0, 1] as k0 2^-20 + k1 2^-43 + k2 2^-56, each rounded to nearest:
// adding a constant leaves the integer in the last bits of the sum.  (Two pieces
// would count what is below 2^-44 as nothing: a long vocabulary beside one token
// that was all but certain.)
struct Pieces {
  uint32_t k0 = 0, k1 = 0, k2 = 0;
  __device__ __forceinline__ void add(float x0, float x1) {
    const uint64_t x = pack2(x0, x1);
    const uint64_t a = add2(x, pack2(12.f, 12.f));  // 2^3 .. 2^4: steps of 2^-20
    const uint64_t d = fma2(add2(a, pack2(-12.f, -12.f)), pack2(-1.f, -1.f), x);  // at most 2^-21, exact
    const uint64_t b = add2(d, pack2(0x1.8p-20f, 0x1.8p-20f));                    // steps of 2^-43
    const uint64_t r = fma2(add2(b, pack2(-0x1.8p-20f, -0x1.8p-20f)), pack2(-1.f, -1.f), d);  // at most 2^-44, exact
    const uint64_t f = add2(r, pack2(0x1.8p-33f, 0x1.8p-33f));                    // steps of 2^-56
    float a0, a1, b0, b1, f0, f1;
    unpack2(a, a0, a1);
    unpack2(b, b0, b1);
    unpack2(f, f0, f1);
    k0 += __float_as_uint(a0) + __float_as_uint(a1) - 2 * __float_as_uint(12.f);
    k1 += __float_as_uint(b0) + __float_as_uint(b1) - 2 * __float_as_uint(0x1.8p-20f);
    k2 += __float_as_uint(f0) + __float_as_uint(f1) - 2 * __float_as_uint(0x1.8p-33f);
  }
  // 56 bits behind the point (up to 512 numbers: |k1| and |k2| stay below 2^31)
  __device__ __forceinline__ uint64_t sum() const {
    return (static_cast<uint64_t>(k0) << (kShift - 20)) +
           static_cast<uint64_t>(static_cast<int64_t>(static_cast<int32_t>(k1)) << (kShift - 43)) +
           static_cast<uint64_t>(static_cast<int64_t>(static_cast<int32_t>(k2)));
  }
};
__device__ __forceinline__ uint64_t pieces(float x) {
  Pieces k;
  k.add(x, 0.f);
  return k.sum();
}

// c as two floats: off by at most 2^-49 of it (from 2^8 on its last 8 bits are
// dropped first, 2^-56 of it).
__device__ __forceinline__ void split_c(Wide c, float &c0, float &c1) {
  const bool large = (c >> 64) != 0;
  const uint64_t x = static_cast<uint64_t>(large ? c >> 8 : c);
  const float unit = large ? 0x1p-48f : 0x1p-56f;
  c0 = __ull2float_rn(x);
  c1 = __ll2float_rn(static_cast<int64_t>(x - __float2ull_rn(c0))) * unit;
  c0 *= unit;
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
  uint64_t total[2][kMaxCluster];  // per pass parity: every CTA's sum
  uint64_t scan[kWarps];
  int32_t path[kMaxNodes], gone[kMaxNodes];  // accepted nodes; tokens removed at the current node
  // the walk, written by thread 0
  int32_t cur, next, n_path, n_gone, again;
  uint64_t s;
  Wide c, c_pass;  // that of the distribution now, that of the next pass
  int32_t kind;    // the next pass's c: 0, 1, or another (2)
  float c0, c1;    // the same as two floats
  int32_t bad;
  int32_t slice;   // the drawn token's warp slice in this CTA, or -1
  uint64_t target;  // what is left of the draw there
};

// The CTA's slices of a node's two rows in shared memory, so that the passes
// after a node's first, and the draw, need not go to memory again.
template <typename T>
struct Kept {
  T *p, *q;  // null: the slices are too long
  int y0;    // the CTA's first position
};
__device__ __forceinline__ void put4(float *to, const float (&x)[4]) {
  *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void put4(__nv_bfloat16 *to, const float (&x)[4]) {  // (bf16 values: exact)
  *reinterpret_cast<uint2 *>(to) =
      make_uint2(__float_as_uint(x[0]) >> 16 | (__float_as_uint(x[1]) & 0xffff0000u),
                 __float_as_uint(x[2]) >> 16 | (__float_as_uint(x[3]) & 0xffff0000u));
}

// What is left of four tokens, in place of x; the same added to a sum.
template <bool kFirst, bool kDraft>
__device__ __forceinline__ void left4(float (&x)[4], const float (&z)[4], float c0, float c1) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    if (kDraft) {
      left2<kFirst>(x[e], x[e + 1], c0, c1, z[e], z[e + 1]);
    } else {
      x[e] = __saturatef(x[e]);
      x[e + 1] = __saturatef(x[e + 1]);
    }
  }
}
template <bool kFirst, bool kDraft>
__device__ __forceinline__ void add4(Pieces &k, float (&x)[4], const float (&z)[4], float c0, float c1) {
  left4<kFirst, kDraft>(x, z, c0, c1);
  k.add(x[0], x[1]);
  k.add(x[2], x[3]);
}

// N steps of 128 positions, all of their loads first.  kFrom: memory (0), the
// same and kept (1), what was kept (2).
template <typename T, bool kFirst, bool kDraft, int kFrom, int N>
__device__ __forceinline__ void steps(const Row<T> &p, const Row<T> &q, const Kept<T> &kept, float c0, float c1, int y,
                                      Pieces &k) {
  float x[N][4], z[kDraft ? N : 1][4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = y + 128 * i;
    four(kFrom == 2 ? kept.p + (at - kept.y0) : p.at + at, x[i]);
    if constexpr (kDraft) four(kFrom == 2 ? kept.q + (at - kept.y0) : q.at + at, z[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (kFrom == 1) {
      put4(kept.p + (y + 128 * i - kept.y0), x[i]);
      if constexpr (kDraft) put4(kept.q + (y + 128 * i - kept.y0), z[i]);
    }
    add4<kFirst, kDraft>(k, x[i], z[kDraft ? i : 0], c0, c1);
  }
}

// One pass over a warp's slice [y0, y1): the sum of max(p - c q, 0), or of p.
// (60 instructions an element with 64-bit integers throughout, and the
// instructions were what a pass took; about 15 so.)
template <typename T, bool kFirst, bool kDraft, int kFrom>
__device__ __forceinline__ uint64_t slice_sum(const Row<T> &p, const Row<T> &q, const Kept<T> &kept, float c0, float c1,
                                              int y0, int y1, int lane) {
  uint64_t sum = 0;
  for (int yb = y0; yb < y1; yb += 128 * 64) {  // (512 elements a lane at most)
    Pieces k;
    const int stop = min(y1, yb + 128 * 64);
    int y = yb + 4 * lane;
    // Inside the row and with both rows alike in memory, plain vector loads:
    // up to eight steps' are under way together.
    if (kFrom == 2 || (yb >= p.off && (!kDraft || p.off == q.off))) {
      int left = kFrom == 2 ? (stop - yb + 127) / 128 : (min(stop, p.end) - yb) / 128;
      for (; left >= 8; left -= 8, y += 1024) steps<T, kFirst, kDraft, kFrom, 8>(p, q, kept, c0, c1, y, k);
      if (left & 4) steps<T, kFirst, kDraft, kFrom, 4>(p, q, kept, c0, c1, y, k), y += 512;
      if (left & 2) steps<T, kFirst, kDraft, kFrom, 2>(p, q, kept, c0, c1, y, k), y += 256;
      if (left & 1) steps<T, kFirst, kDraft, kFrom, 1>(p, q, kept, c0, c1, y, k), y += 128;
    }
    if (kFrom < 2)
      for (; y - 4 * lane < stop; y += 128) {  // (whole steps: what is kept ends with zeros)
        float x[4], z[4];
        load_p(p, y, x);
        if (kDraft) load_q(p, q, y, z);
        if (kFrom == 1) {
          put4(kept.p + (y - kept.y0), x);
          if (kDraft) put4(kept.q + (y - kept.y0), z);
        }
        add4<kFirst, kDraft>(k, x, z, c0, c1);
      }
    sum += k.sum();
  }
  return sum;
}
template <typename T, bool kFirst, bool kDraft>
__device__ __forceinline__ uint64_t slice_sum_from(int from, const Row<T> &p, const Row<T> &q, const Kept<T> &kept, float c0,
                                                   float c1, int y0, int y1, int lane) {
  return from == 0   ? slice_sum<T, kFirst, kDraft, 0>(p, q, kept, c0, c1, y0, y1, lane)
         : from == 1 ? slice_sum<T, kFirst, kDraft, 1>(p, q, kept, c0, c1, y0, y1, lane)
                     : slice_sum<T, kFirst, kDraft, 2>(p, q, kept, c0, c1, y0, y1, lane);
}

// Positions of a warp's slice: whole steps of 128 (a lane's 4 x 32 lanes).
__host__ __device__ __forceinline__ int slice_length(int vocab, int slices) {
  return ((vocab + 3 + slices - 1) / slices + 127) / 128 * 128;
}

template <typename T, int kCluster>
__global__ void __launch_bounds__(kThreads) tree_verify_kernel(const __grid_constant__ TreeVerifyArgs a) {
  constexpr int kSlices = kCluster * kWarps;
  extern __shared__ __align__(16) uint8_t kept_raw[];
  __shared__ Smem S;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  // Shared memory of another CTA may be touched only once that CTA is known to
  // run: arrive here, wait behind the loads of the single values, which hide it.
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const int r = blockIdx.x / kCluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TN = a.max_nodes, V = a.vocab, n = a.n_nodes[r];
  const T *p0 = static_cast<const T *>(a.p) + static_cast<int64_t>(r) * TN * a.p_stride;
  const T *q0 = a.q ? static_cast<const T *>(a.q) + static_cast<int64_t>(r) * TN * a.q_stride : nullptr;
  int par = -2, tok = 0;
  float ua = 0.f;
  if (tid < TN) {  // (beside the load of n)
    const int64_t at = static_cast<int64_t>(r) * TN + tid;
    par = a.parent[at];
    tok = a.token[at];
    ua = a.u_accept[at];
  }
  const float us = a.u_sample[r];
  if (tid == 0) S.bad = n < 0 || n > TN;
  __syncthreads();
  if (!S.bad && tid < n) {
    S.token[tid] = tok;
    const bool root = tid == 0;
    if (par < -1 || par >= tid || (!root && (tok < 0 || tok >= V))) {
      S.bad = 1;
    } else if (par >= 0) {
      S.px[tid] = to_fix(one(p0 + par * a.p_stride + tok));
      S.qx[tid] = q0 ? to_fix(one(q0 + par * a.q_stride + tok)) : kOne;
      S.u[tid] = to_fix(ua);
    }
  }
  if (tid < kMaxNodes) S.parent[tid] = tid < n ? par : -2;
  __syncthreads();
  asm volatile("barrier.cluster.wait;" ::: "memory");
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
  const int per = slice_length(V, kSlices);
  Kept<T> kept = {nullptr, nullptr, rank * kWarps * per};
  if (a.keep) {
    kept.p = reinterpret_cast<T *>(kept_raw);
    kept.q = kept.p + kWarps * per;
  }
  int kept_p = -1, kept_q = -1;  // the nodes whose rows are kept
  int parity = 0;
  bool fresh = false;  // the slices' sums are those of (cur, c)
  for (;;) {
    if (warp == 0) {
      // on to the next rejection that needs a sum, or to the end: the whole
      // warp walks, its lanes looking for a node's next child
      int cur = S.cur, i = S.next, n_path = S.n_path, n_gone = S.n_gone, again = 0;
      Wide c = S.c;
      uint64_t s = S.s;
      bool moved = false;
      while (!again) {
        int x = kMaxNodes;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          const unsigned hit = __ballot_sync(0xffffffffu, S.parent[32 * k + lane] == cur && 32 * k + lane >= i);
          if (hit) x = 32 * k + __ffs(hit) - 1;
        }
        if (x == kMaxNodes) {
          i = n;
          break;
        }
        i = x + 1;
        uint64_t rest = left_of(S.px[x], c, S.qx[x]);
        if (!q0) {
          bool gone = false;
          for (int j = lane; j < n_gone; j += 32) gone |= S.gone[j] == S.token[x];
          rest = __any_sync(0xffffffffu, gone) ? 0 : S.px[x];
        }
        if (mul_fix(mul_fix(S.u[x], S.qx[x]), s) < rest) {
          cur = x;
          if (lane == 0) S.path[n_path] = x;
          ++n_path;
          n_gone = 0;
          c = 0;
          s = kOne;
          moved = true;
        } else if (!q0) {
          if (rest > 0) {
            if (lane == 0) S.gone[n_gone] = S.token[x];
            ++n_gone;
            __syncwarp();
          }
          s = s > rest ? s - rest : 0;
          moved = true;
        } else {
          again = 1;
        }
      }
      if (lane == 0) {
        S.cur = cur;
        S.next = i;
        S.n_path = n_path;
        S.n_gone = n_gone;
        S.c = c;
        S.s = s;
        S.again = again | (moved ? 2 : 0);
        const Wide pass = again ? c + s : c;
        S.c_pass = pass;
        S.kind = pass == 0 ? 0 : pass == kOne ? 1 : 2;
        // (64-bit conversions run at a sixteenth of the rate: one thread's)
        split_c(pass, S.c0, S.c1);
      }
    }
    __syncthreads();
    const int again = S.again;
    if (again & 2) fresh = false;
    if (!(again & 1) && fresh) break;
    // one pass: the slices' sums of max(p - c q, 0)
    const int kind = S.kind;
    const Row<T> p(p0 + S.cur * a.p_stride, V);
    uint64_t sum = 0;
    const int y0 = (rank * kWarps + warp) * per, y1 = min(y0 + per, p.end);
    if (kind == 0) {
      const int from = !a.keep ? 0 : kept_p == S.cur ? 2 : 1;
      sum = slice_sum_from<T, false, false>(from, p, p, kept, 0.f, 0.f, y0, y1, lane);
      if (from == 1) kept_p = S.cur, kept_q = -1;
    } else {
      const Row<T> q(q0 + S.cur * a.q_stride, V);
      const float c0 = S.c0, c1 = S.c1;
      const int from = !a.keep ? 0 : kept_q == S.cur ? 2 : 1;
      sum = kind == 1 ? slice_sum_from<T, true, true>(from, p, q, kept, c0, c1, y0, y1, lane)
                      : slice_sum_from<T, false, true>(from, p, q, kept, c0, c1, y0, y1, lane);
      if (from == 1) kept_p = kept_q = S.cur;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) S.wsum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      if (S.n_gone > 0) {  // tokens removed at this node
        if (lane == 0)
          for (int j = 0; j < S.n_gone; ++j) {
            const int y = S.gone[j] + p.off, w = y / per - rank * kWarps;
            if (w >= 0 && w < kWarps) S.wsum[w] -= pieces(__saturatef(one(p.at + y)));
          }
        __syncwarp();
      }
      uint64_t t = lane < kWarps ? S.wsum[lane] : 0;
#pragma unroll
      for (int o = kWarps / 2; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      t = __shfl_sync(0xffffffffu, t, 0);
      if (lane < kCluster) cluster.map_shared_rank(&S, lane)->total[parity][rank] = t;
    }
    cluster.sync();
    if (again & 1) {
      uint64_t t = 0;
#pragma unroll
      for (int x = 0; x < kCluster; ++x) t += S.total[parity][x];
      fresh = t > 0;  // nothing left: the distribution before the rejection stays
      __syncthreads();
      if (tid == 0 && t > 0) {
        S.c = S.c_pass;
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
      uint64_t t = mul_fix(to_fix(us), all);
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
  const int kind = S.kind;  // (the last pass's c is the one that stays)
  const float c0 = S.c0, c1 = S.c1;
  uint64_t target = S.target;
  for (int yb = y0; yb < y1; yb += 4 * kThreads) {
    const int y = yb + 4 * tid;
    uint64_t v[4] = {0, 0, 0, 0}, mine = 0;
    if (y < y1) {
      float x[4], z[4] = {0.f, 0.f, 0.f, 0.f};
      if (kept_p == S.cur) four(kept.p + (y - kept.y0), x);
      else load_p(p, y, x);
      if (kind != 0) {
        const Row<T> q(q0 + S.cur * a.q_stride, V);
        if (kept_q == S.cur) four(kept.q + (y - kept.y0), z);
        else load_q(p, q, y, z);
      }
      if (kind == 0) left4<true, false>(x, z, c0, c1);
      else if (kind == 1) left4<true, true>(x, z, c0, c1);
      else left4<false, true>(x, z, c0, c1);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = pieces(x[e]);
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

namespace {
constexpr size_t kMostKept = 200 * 1024;  // of a CTA's shared memory

template <typename T, int kCluster>
cudaError_t launch(TreeVerifyArgs a, cudaStream_t s) {
  static bool configured = false;
  if (!configured) {
    cudaError_t e = cudaFuncSetAttribute(tree_verify_kernel<T, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kMostKept));
    if (e == cudaSuccess && kCluster > 8)
      e = cudaFuncSetAttribute(tree_verify_kernel<T, kCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured = true;
  }
  const size_t kept = static_cast<size_t>(slice_length(a.vocab, kCluster * kWarps)) * kWarps * sizeof(T) * (a.q ? 2 : 1);
  a.keep = kept <= kMostKept;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows) * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.keep ? kept : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<T, kCluster>, a);
}
template <typename T>
cudaError_t launch(const TreeVerifyArgs &a, cudaStream_t s) {
  // Sixteen CTAs a row while all rows' run at once, two on an SM (4 rows of
  // 131072 fp32: 11.0 us, with eight a tenth more), else eight (64 rows in
  // bf16: 22.8 us in two waves; with four 28.0 in one, and with CTAs of 256
  // threads, sixteen a row and all rows at once, 24.3; all measured with sums of
  // 43 bits, which took 0.4 to 2 us less).
  return a.n_rows * 16 <= 2 * device_sm_count() ? launch<T, 16>(a, s) : launch<T, 8>(a, s);
}
}  // namespace

cudaError_t launch_tree_verify(const TreeVerifyArgs &a, cudaStream_t s) {
  return a.dtype == HW_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace hw
