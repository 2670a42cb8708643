// cache_ops.cu - tokens written into a cache and read back (hw_cache_write,
// hw_cache_read), finished steps committed between 4-bit caches
// (hw_block_commit_many_fp4).
//
//   write: K[l][h][slot] = store(rho(k_new[l][i][h], pos)),  V[l][h][slot] = store(v_new[l][i][h])
//   read:  k_out[l][i][h] = value(K[l][h][slot]),  v_out alike
//   commit: K_dst = store(rho(value(K_src), delta)), V_dst = V_src
//
// Writes and reads are bound by DRAM: every element is read once and written once, a
// thread holds 16 bytes of the first half of a row and the 16 of the second
// that they turn with, so a rotation needs no exchange, and a 4-bit row's maximum is
// three shuffles among its 8 threads.  Cosines and sines are made once for a
// CTA's tokens in shared memory and serve all its layers and heads (a commit's, once a
// range: all its tokens turn by the same angle).  Measured, a long prompt's tokens in 4 bits
// (675 MB): written in 131 us, 5.2 TB/s, read in 124 us, 5.5 TB/s.
#include <cuda_fp8.h>

#include <type_traits>

#include "hw_cache.h"
#include "hw_device.cuh"
#include "hw_fp4.cuh"
#include "hw_rope_exact.cuh"

namespace hw {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // a CTA's tokens (of hw_cache_write)

struct E4M3 {
  uint8_t code;
};
struct E2M1x2 {
  uint8_t codes;
};

// What a cache of type Store takes and gives.
template <typename Store>
struct Format {
  using Act = __nv_bfloat16;
};
template <>
struct Format<float> {
  using Act = float;
};

// 16 bytes of activations as fp32 and back.
template <typename Act>
struct Vec {
  static constexpr int N = 16 / sizeof(Act);
  __device__ __forceinline__ static void unpack(const uint4 &w, float *x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 4) {
        x[i] = __uint_as_float(v[i]);
      } else {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ static uint4 pack(const float *x) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 4) {
        v[i] = __float_as_uint(x[i]);
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t *>(&p);
      }
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};

__device__ __forceinline__ uint32_t e4m3x4(const float *x) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ void e4m3x4_values(uint32_t w, float *x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i) & 0xffffu), __NV_E4M3));
    const float2 f = __half22float2(h);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// 8 elements of a row's first half and the 8 that they turn with.
__device__ __forceinline__ void turn8(const float (&x0)[8], const float (&x1)[8], const float (&cs)[8],
                                      const float (&sn)[8], float (&y0)[8], float (&y1)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float2 a, b;
    fp4_turn2(make_float2(x0[e], x0[e + 1]), make_float2(x1[e], x1[e + 1]), make_float2(cs[e], cs[e + 1]),
              make_float2(sn[e], sn[e + 1]), a, b);
    y0[e] = a.x;
    y0[e + 1] = a.y;
    y1[e] = b.x;
    y1[e + 1] = b.y;
  }
}

// The codes of x[] / s as quotient() has them, 8 bytes.
__device__ __forceinline__ uint2 e4m3_quotients(const float (&x)[8], float s, float inv) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 q = __fmul2_rn(make_float2(x[j], x[j + 1]), make_float2(inv, inv));
    const float2 r = __ffma2_rn(q, make_float2(-s, -s), make_float2(x[j], x[j + 1]));
    const float2 z = __ffma2_rn(r, make_float2(inv, inv), q);
    y[j] = fabsf(q.x) < INFINITY ? z.x : q.x;
    y[j + 1] = fabsf(q.y) < INFINITY ? z.y : q.y;
  }
  return make_uint2(e4m3x4(y), e4m3x4(y + 4));
}

// Rows of a CTA's tokens: (layer, token, kv head), 8 or so threads each.  blockIdx.x: the
// tokens, blockIdx.y: a share of the layers.
template <typename Store, int D>
__global__ void __launch_bounds__(kThreads, 3) cache_write_kernel(const __grid_constant__ CacheArgs a) {
  using Act = typename Format<Store>::Act;
  constexpr bool kFp4 = std::is_same_v<Store, E2M1x2>;
  constexpr int N = Vec<Act>::N, kPer = D / 2 / N;  // threads a row
  __shared__ float2 turn[kTokens][D / 2];
  __shared__ int32_t slots[kTokens];
  __shared__ float2 table[kFp4 ? 65 : 1];
  const int tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(kTokens), a.n_tokens - t0));
  if (tid < nt) {
    int32_t s = __ldg(a.slot + t0 + tid);
    if (s < -1 || s >= a.capacity) {
      if (a.flags && blockIdx.y == 0) flag_error(a.flags, HW_DEV_BAD_RANGE);
      s = -1;
    }
    slots[tid] = s;
  }
  if constexpr (kFp4) {
    if (tid >= 64 && tid < 129) table[tid - 64] = kSin256[tid - 64];
    __syncthreads();
  }
  for (int i = tid; i < nt * (D / 2); i += kThreads) {
    const int t = i / (D / 2), j = i % (D / 2);
    const int64_t p = __ldg(a.pos + t0 + t);
    float c, s;
    if constexpr (kFp4)
      rope_cos_sin_exact(p, a.phase[j], &c, &s, table);
    else if constexpr (sizeof(Store) == 1)
      rope_cos_sin_near(p, a.phase[j], &c, &s);
    else
      rope_cos_sin(p, a.phase[j], &c, &s);
    turn[t][j] = make_float2(c, s);
  }
  __syncthreads();
  const int H = a.n_kv_heads;
  const int l0 = static_cast<int>(static_cast<int64_t>(a.n_layers) * blockIdx.y / gridDim.y);
  const int l1 = static_cast<int>(static_cast<int64_t>(a.n_layers) * (blockIdx.y + 1) / gridDim.y);
  const int parts = nt * H * kPer;
  const int64_t from_step = static_cast<int64_t>(a.n_tokens) * H * D, row_step = static_cast<int64_t>(H) * a.capacity;
  // A thread's part of a row in one layer after the other: its place and its angles are
  // the same in all of them.  The next layer's loads run under this one's arithmetic (without
  // that, 32 warps of 64 bytes a thread, it reached 4.4 TB/s).  (Whole warps: the rows'
  // threads shuffle.)
  for (int base = 0; base < parts; base += kThreads) {
    const bool in = base + tid < parts;
    const int r = in ? base + tid : 0;
    const int c = r % kPer, th = r / kPer, h = th / nt, t = th - h * nt;  // (neighbours in the cache side by side)
    const int32_t slot = slots[t];
    const bool on = in && slot >= 0;
    int64_t from = ((static_cast<int64_t>(l0) * a.n_tokens + t0 + t) * H + h) * D + c * N;
    int64_t row = (static_cast<int64_t>(l0) * H + h) * a.capacity + (on ? slot : 0);
    float cs[N], sn[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      cs[j] = turn[t][c * N + j].x;
      sn[j] = turn[t][c * N + j].y;
    }
    uint4 next[4] = {};
    auto load = [&]() {
      const Act *kn = static_cast<const Act *>(a.k_new) + from, *vn = static_cast<const Act *>(a.v_new) + from;
      next[0] = __ldg(reinterpret_cast<const uint4 *>(kn));
      next[1] = __ldg(reinterpret_cast<const uint4 *>(kn + D / 2));
      next[2] = __ldg(reinterpret_cast<const uint4 *>(vn));
      next[3] = __ldg(reinterpret_cast<const uint4 *>(vn + D / 2));
      from += from_step;
    };
    if (on && l0 < l1) load();
    for (int l = l0; l < l1; ++l, row += row_step) {
      const uint4 raw[4] = {next[0], next[1], next[2], next[3]};
      if (on && l + 1 < l1) load();
      float x0[N], x1[N], k0[N], k1[N], v0[N], v1[N];
      Vec<Act>::unpack(raw[0], x0);
      Vec<Act>::unpack(raw[1], x1);
      Vec<Act>::unpack(raw[2], v0);
      Vec<Act>::unpack(raw[3], v1);
      if constexpr (kFp4) {
        turn8(x0, x1, cs, sn, k0, k1);
      } else {  // as the appends of the decode calls
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const float2 p = make_float2(x0[j], x0[j + 1]), q = make_float2(x1[j], x1[j + 1]);
          const float2 c = make_float2(cs[j], cs[j + 1]), s = make_float2(sn[j], sn[j + 1]);
          const float2 m = __fmul2_rn(q, s);
          const float2 y0 = __ffma2_rn(p, c, make_float2(-m.x, -m.y)), y1 = __ffma2_rn(q, c, __fmul2_rn(p, s));
          k0[j] = y0.x;
          k0[j + 1] = y0.y;
          k1[j] = y1.x;
          k1[j + 1] = y1.y;
        }
      }
      if constexpr (kFp4) {
        uint32_t kl, kh, vl, vh;
        const float ks = fp4_row<false>(k0, k1, kl, kh);
        const float vs = fp4_row<true>(v0, v1, vl, vh);
        if (on) {
          uint32_t *kd = static_cast<uint32_t *>(a.k_cache) + row * (D / 8) + c;
          uint32_t *vd = static_cast<uint32_t *>(a.v_cache) + row * (D / 8) + c;
          kd[0] = kl;
          kd[D / 16] = kh;
          vd[0] = vl;
          vd[D / 16] = vh;
          if (c == 0) static_cast<uint32_t *>(a.kv_scale)[row] = fp4_scale_word(ks, vs);
        }
      } else if (on) {
        Store *kd = static_cast<Store *>(a.k_cache) + row * D + c * N;
        Store *vd = static_cast<Store *>(a.v_cache) + row * D + c * N;
        if constexpr (sizeof(Store) == 1) {  // E4M3
          const float ks = __ldg(a.k_scale + l * H + h), vs = __ldg(a.v_scale + l * H + h);
          const float ki = reciprocal(ks), vi = reciprocal(vs);
          // (5003 tokens: 14.3 us, with the division of the language 18.6, with products by 1 / s 12.9)
          *reinterpret_cast<uint2 *>(kd) = e4m3_quotients(k0, ks, ki);
          *reinterpret_cast<uint2 *>(kd + D / 2) = e4m3_quotients(k1, ks, ki);
          *reinterpret_cast<uint2 *>(vd) = e4m3_quotients(v0, vs, vi);
          *reinterpret_cast<uint2 *>(vd + D / 2) = e4m3_quotients(v1, vs, vi);
        } else {
          *reinterpret_cast<uint4 *>(kd) = Vec<Act>::pack(k0);
          *reinterpret_cast<uint4 *>(kd + D / 2) = Vec<Act>::pack(k1);
          *reinterpret_cast<uint4 *>(vd) = Vec<Act>::pack(v0);
          *reinterpret_cast<uint4 *>(vd + D / 2) = Vec<Act>::pack(v1);
        }
      }
    }
  }
}

// Rows (layer, token, kv head) in the order of the outputs.
template <typename Store, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a) {
  using Act = typename Format<Store>::Act;
  constexpr bool kFp4 = std::is_same_v<Store, E2M1x2>;
  constexpr int N = Vec<Act>::N, kPer = D / N;  // threads a row, 16 bytes of output each
  const int H = a.n_kv_heads;
  const int64_t rows = static_cast<int64_t>(a.n_layers) * a.n_tokens * H, end = rows * kPer;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < end;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int c = static_cast<int>(i % kPer);
    const int64_t lth = i / kPer, lt = div_nn(lth, H);
    const int h = static_cast<int>(lth - lt * H);
    const int64_t l = div_nn(lt, a.n_tokens), t = lt - l * a.n_tokens;
    const int32_t slot = __ldg(a.slot + t);
    if (slot < 0 || slot >= a.capacity) {
      if (slot != -1 && c == 0 && h == 0 && l == 0 && a.flags) flag_error(a.flags, HW_DEV_BAD_RANGE);
      continue;
    }
    const int64_t row = (l * H + h) * a.capacity + slot;
    uint4 ko, vo;
    if constexpr (kFp4) {
      const uint32_t kw = __ldg(reinterpret_cast<const uint32_t *>(a.k_cache) + row * (D / 8) + c);
      const uint32_t vw = __ldg(reinterpret_cast<const uint32_t *>(a.v_cache) + row * (D / 8) + c);
      const uint32_t sw = __ldg(static_cast<const uint32_t *>(a.kv_scale) + row);
      float k[8], v[8];
      fp4_levels8(kw, k);
      fp4_levels8(vw, v);
      const float ks = fp4_k_scale(sw), vs = fp4_v_scale(sw);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[j] *= ks;
        v[j] *= vs;
      }
      ko = Vec<Act>::pack(k);
      vo = Vec<Act>::pack(v);
    } else if constexpr (sizeof(Store) == 1) {
      const uint2 kw = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.k_cache) + row * D) + c);
      const uint2 vw = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.v_cache) + row * D) + c);
      const float ks = __ldg(a.k_scale + l * H + h), vs = __ldg(a.v_scale + l * H + h);
      float k[8], v[8];
      e4m3x4_values(kw.x, k);
      e4m3x4_values(kw.y, k + 4);
      e4m3x4_values(vw.x, v);
      e4m3x4_values(vw.y, v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[j] *= ks;
        v[j] *= vs;
      }
      ko = Vec<Act>::pack(k);
      vo = Vec<Act>::pack(v);
    } else {
      ko = __ldg(reinterpret_cast<const uint4 *>(static_cast<const Store *>(a.k_cache) + row * D) + c);
      vo = __ldg(reinterpret_cast<const uint4 *>(static_cast<const Store *>(a.v_cache) + row * D) + c);
    }
    __stcs(static_cast<uint4 *>(a.k_out) + i, ko);
    __stcs(static_cast<uint4 *>(a.v_out) + i, vo);
  }
}

// Finished steps of 4-bit caches, in tiles of 64 tokens of one range and (layer, kv head): 4 KB
// of key codes, 4 KB of value codes and 64 scales, each contiguous.  A CTA has an equal,
// contiguous share of all tiles.  Bytes are few here (264 a token read and written) beside what a
// turned key costs, so instructions bound it, and the layout is the one with the fewest:
//  - 4 threads a token, 32 elements each, its key's and value's 16-byte pieces copied ahead by
//    the thread that uses them (three tiles, 24 KB a CTA), so no thread waits for another's;
//  - what goes together in a turn is brought together by 2 shuffles, and taken back by 2.
// A model's 233 MB: 56 us, 4.2 TB/s, 68 % of the issue slots, 59 % of the integer pipe, which
// also converts codes.  (Before: 8 threads a token with loads into registers, 71 us; keys
// through shared memory between barriers, 61 us; 3 CTAs an SM, 5 or 6 tiles ahead: 56 to 58.)
constexpr int kCommitRows = kThreads / 4, kCommitStages = 4, kCommitCtas = 2;  // (CTAs an SM)

struct CommitTile {
  uint4 k[kThreads], v[kThreads];  // a thread's 16 bytes of its token's 64
  uint32_t s[kThreads];            // and its copy of the token's scales
};

__device__ __forceinline__ void copy_16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src)
               : "memory");
}

// A place among the tiles: range, row (layer, kv head), first token in the range.
struct CommitWalk {
  int c, j;
  int64_t lh, rows;
  __device__ CommitWalk(const CommitArgs &a, int64_t tile) : rows(static_cast<int64_t>(a.n_layers) * a.n_kv_heads) {
    for (c = 0; c < a.n_commits; ++c) {
      const int64_t in_row = (static_cast<int64_t>(a.n_tokens[c]) + kCommitRows - 1) / kCommitRows, n = in_row * rows;
      if (tile < n) {
        lh = tile / in_row;
        j = static_cast<int>(tile - lh * in_row) * kCommitRows;
        return;
      }
      tile -= n;
    }
  }
  __device__ __forceinline__ void next(const CommitArgs &a) {  // (there is one)
    if (a.n_tokens[c] - j > kCommitRows) {
      j += kCommitRows;
      return;
    }
    j = 0;
    if (++lh < rows) return;
    lh = 0;
    while (++c < a.n_commits && a.n_tokens[c] == 0) {
    }
  }
  __device__ __forceinline__ int tokens(const CommitArgs &a) const { return min(a.n_tokens[c] - j, kCommitRows); }
  __device__ __forceinline__ int64_t src(const CommitArgs &a) const { return lh * a.src_capacity + a.src_begin[c] + j; }
  __device__ __forceinline__ int64_t dst(const CommitArgs &a) const { return lh * a.dst_capacity + a.dst_offset[c] + j; }
};

// 16 pairs of levels turned (e0, e1: 2 words of codes each, in place), and the largest magnitude.
__device__ __forceinline__ float turn_levels(const uint32_t (&e0)[2], const uint32_t (&e1)[2], const float (&cs)[16],
                                             const float (&sn)[16], float (&y0)[16], float (&y1)[16]) {
  float top = 0.f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float x0[8], x1[8];
    fp4_levels8(e0[w], x0);
    fp4_levels8(e1[w], x1);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int i = 8 * w + e;
      const float2 p = make_float2(x0[e], x0[e + 1]), q = make_float2(x1[e], x1[e + 1]);
      const float2 c = make_float2(cs[i], cs[i + 1]), n = make_float2(sn[i], sn[i + 1]);
      const float2 a = __ffma2_rn(q, make_float2(-n.x, -n.y), __fmul2_rn(p, c));
      const float2 b = __ffma2_rn(p, n, __fmul2_rn(q, c));
      y0[i] = a.x;
      y0[i + 1] = a.y;
      y1[i] = b.x;
      y1[i + 1] = b.y;
      top = max3_abs_nan(max3_abs_nan(top, a.x, a.y), b.x, b.y);
    }
  }
  return top;
}
__device__ __forceinline__ void codes_of(const float (&y)[16], float r, uint32_t (&e)[2]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 a = __fmul2_rn(make_float2(y[8 * w + k], y[8 * w + k + 1]), make_float2(r, r));
      t[k] = a.x;
      t[k + 1] = a.y;
    }
    e[w] = e2m1x8(t);
  }
}

// A token's key, 32 elements from 32 (tid & 3) on in each of 4 neighbouring threads, turned and
// encoded again; its new scale is the result.  The threads two apart hold what turns
// together: they exchange 16 elements, so that either has 16 pairs, and exchange them back.
// Levels are turned as they are (the scale is a factor of all), in fp32 with fused products, and
// encoded by one product with s / next: the code is the nearest one but where the quotient lies
// within 2^-21 of a border, as near as the turn's own roundings are.  Numbers that the turn
// leaves alone (slow pairs, with nothing to turn in) can stand on a border.  s / next is rounded
// to nearest for them: n / m rounded, times m, is n for every m = 2^i + 2^j (W. Kahan), which levels
// are, so a border is met exactly and goes to the even code.  (With every code decided exactly from
// scaled, unfused products a model's commit takes 71 us, not 56.)
__device__ __forceinline__ float commit_key(uint4 &k, const float (&cs)[16], const float (&sn)[16], float s) {
  const bool up = threadIdx.x & 2;
  auto other = [](uint32_t x) { return __shfl_xor_sync(0xffffffffu, x, 2); };
  uint32_t e0[2], e1[2];
  {
    const uint32_t g0 = other(up ? k.x : k.z), g1 = other(up ? k.y : k.w);
    e0[0] = up ? g0 : k.x;
    e0[1] = up ? g1 : k.y;
    e1[0] = up ? k.z : g0;
    e1[1] = up ? k.w : g1;
  }
  float y0[16], y1[16];
  float top = turn_levels(e0, e1, cs, sn, y0, y1);
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const float next = fp4_scale(top * s);
  if (next > 0.f) {
    const float r = __fdiv_rn(s, next);
    codes_of(y0, r, e0);
    codes_of(y1, r, e1);
  } else {
    e0[0] = e0[1] = e1[0] = e1[1] = 0;
  }
  const uint32_t g0 = other(up ? e0[0] : e1[0]), g1 = other(up ? e0[1] : e1[1]);
  k = up ? make_uint4(g0, g1, e1[0], e1[1]) : make_uint4(e0[0], e0[1], g0, g1);
  return next;
}

__global__ void __launch_bounds__(kThreads, kCommitCtas)
    commit_fp4_kernel(const __grid_constant__ CommitArgs a, const CommitScales scales, int64_t n_tiles) {
  __shared__ CommitTile ring[kCommitStages];
  __shared__ float2 turn[64];
  const int tid = threadIdx.x, row = tid >> 2;
  const int64_t t0 = n_tiles * blockIdx.x / gridDim.x, t1 = n_tiles * (blockIdx.x + 1) / gridDim.x;
  CommitWalk ld(a, t0), w = ld;
  int64_t left = t1 - t0;  // tiles to be loaded
  auto load = [&](CommitTile &t) {
    if (left > 0) {
      const int64_t so = ld.src(a);
      if (row < ld.tokens(a)) {
        copy_16(&t.k[tid], static_cast<const uint4 *>(a.k_src) + so * 4 + tid);
        copy_16(&t.v[tid], static_cast<const uint4 *>(a.v_src) + so * 4 + tid);
        copy_4(&t.s[tid], scales.src + so + row);
      }
      if (--left > 0) ld.next(a);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kCommitStages - 1; ++i) load(ring[i]);
  float cs[16], sn[16];
  int of = -1;  // the range whose angle they are of
  int st = 0;
  for (int64_t i = t0; i < t1; ++i) {
    if (w.c != of) {  // (all tokens of a range turn by the same angle)
      of = w.c;
      __syncthreads();
      if (tid < 64) rope_cos_sin_exact(a.delta[of], a.phase[tid], &turn[tid].x, &turn[tid].y);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 cst = turn[32 * (tid & 1) + 8 * (tid & 2) + e];
        cs[e] = cst.x;
        sn[e] = cst.y;
      }
    }
    // (a thread uses what it has copied itself: nobody waits for another one)
    asm volatile("cp.async.wait_group %0;" ::"n"(kCommitStages - 2) : "memory");
    const CommitTile &t = ring[st];
    uint4 k = t.k[tid];
    const uint4 v = t.v[tid];
    uint32_t sw = t.s[tid];
    st = st + 1 == kCommitStages ? 0 : st + 1;
    load(ring[(st + kCommitStages - 2) % kCommitStages]);
    if (a.delta[of] != 0) sw = fp4_scale_word(commit_key(k, cs, sn, fp4_k_scale(sw)), fp4_v_scale(sw));
    if (row < w.tokens(a)) {
      const int64_t to = w.dst(a);
      static_cast<uint4 *>(a.k_dst)[to * 4 + tid] = k;
      static_cast<uint4 *>(a.v_dst)[to * 4 + tid] = v;
      if ((tid & 3) == 0) scales.dst[to + row] = sw;
    }
    if (i + 1 < t1) w.next(a);
  }
}

int sm_count() {
  const int n = device_sm_count();
  return n > 0 ? n : 152;
}

template <typename Store, int D>
void write_t(const CacheArgs &a, cudaStream_t s) {
  const int64_t tiles = (static_cast<int64_t>(a.n_tokens) + kTokens - 1) / kTokens;
  // the layers of a tile of tokens in as many CTAs as fill the GPU a few times over
  int64_t split = (8ll * sm_count() + tiles - 1) / tiles;
  if (split > a.n_layers) split = a.n_layers;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(split));
  cache_write_kernel<Store, D><<<grid, kThreads, 0, s>>>(a);
}
template <typename Store, int D>
void read_t(const CacheArgs &a, cudaStream_t s) {
  const int per = D * static_cast<int>(sizeof(typename Format<Store>::Act)) / 16;
  const int64_t work = static_cast<int64_t>(a.n_layers) * a.n_tokens * a.n_kv_heads * per;
  int64_t ctas = (work + kThreads - 1) / kThreads;
  const int64_t most = 16ll * sm_count();
  cache_read_kernel<Store, D><<<static_cast<unsigned>(ctas < most ? ctas : most), kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_cache_write(const CacheArgs &a, int dtype, cudaStream_t s) {
  if (dtype == HW_F32)
    a.head_dim == 64 ? write_t<float, 64>(a, s) : write_t<float, 128>(a, s);
  else if (dtype == HW_BF16)
    a.head_dim == 64 ? write_t<__nv_bfloat16, 64>(a, s) : write_t<__nv_bfloat16, 128>(a, s);
  else if (dtype == HW_FP8_E4M3)
    write_t<E4M3, 128>(a, s);
  else
    write_t<E2M1x2, 128>(a, s);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheArgs &a, int dtype, cudaStream_t s) {
  if (dtype == HW_F32)
    a.head_dim == 64 ? read_t<float, 64>(a, s) : read_t<float, 128>(a, s);
  else if (dtype == HW_BF16)
    a.head_dim == 64 ? read_t<__nv_bfloat16, 64>(a, s) : read_t<__nv_bfloat16, 128>(a, s);
  else if (dtype == HW_FP8_E4M3)
    read_t<E4M3, 128>(a, s);
  else
    read_t<E2M1x2, 128>(a, s);
  return cudaGetLastError();
}

cudaError_t launch_commit_fp4(const CommitArgs &a, const CommitScales &scales, cudaStream_t s) {
  int64_t tiles = 0;
  for (int c = 0; c < a.n_commits; ++c) tiles += (static_cast<int64_t>(a.n_tokens[c]) + kCommitRows - 1) / kCommitRows;
  tiles *= static_cast<int64_t>(a.n_layers) * a.n_kv_heads;
  if (tiles == 0) return cudaSuccess;
  const int64_t most = static_cast<int64_t>(kCommitCtas) * sm_count();
  commit_fp4_kernel<<<static_cast<unsigned>(tiles < most ? tiles : most), kThreads, 0, s>>>(a, scales, tiles);
  return cudaGetLastError();
}

}  // namespace hw
