// cache_ops.cu - tokens written into a cache and read back (hw_cache_write,
// hw_cache_read), finished steps committed between 4-bit caches
// (hw_block_commit_many_fp4).
//
//   write: K[l][h][slot] = store(rho(k_new[l][i][h], pos)),  V[l][h][slot] = store(v_new[l][i][h])
//   read:  k_out[l][i][h] = value(K[l][h][slot]),  v_out alike
//   commit: K_dst = store(rho(value(K_src), delta)), V_dst = V_src
//
// All three are bound by DRAM: every element is read once and written once, a
// thread holds 16 bytes of the first half of a row and the 16 of the second that
// they turn with, so a rotation needs no exchange, and a 4-bit row's maximum is
// three shuffles among its 8 threads.  Cosines and sines are made once for a
// CTA's tokens in shared memory and serve all its layers and heads (a commit's, once a
// CTA: all its tokens turn by the same angle).
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

// Rows of a CTA's tokens: (layer, token, kv head), 8 or so threads each.  blockIdx.x: the
// tokens, blockIdx.y: a share of the layers.
template <typename Store, int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a) {
  using Act = typename Format<Store>::Act;
  constexpr bool kFp4 = std::is_same_v<Store, E2M1x2>;
  constexpr int N = Vec<Act>::N, kPer = D / 2 / N;  // threads a row
  __shared__ float2 turn[kTokens][D / 2];
  __shared__ int32_t slots[kTokens];
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
  for (int i = tid; i < nt * (D / 2); i += kThreads) {
    const int t = i / (D / 2), j = i % (D / 2);
    const int64_t p = __ldg(a.pos + t0 + t);
    float c, s;
    if constexpr (kFp4)
      rope_cos_sin_exact(p, a.phase[j], &c, &s);
    else
      rope_cos_sin(p, a.phase[j], &c, &s);
    turn[t][j] = make_float2(c, s);
  }
  __syncthreads();
  const int H = a.n_kv_heads;
  const int per_layer = nt * H * kPer;
  const int l0 = static_cast<int>(static_cast<int64_t>(a.n_layers) * blockIdx.y / gridDim.y);
  const int l1 = static_cast<int>(static_cast<int64_t>(a.n_layers) * (blockIdx.y + 1) / gridDim.y);
  const int64_t end = static_cast<int64_t>(l1 - l0) * per_layer;
  const Act *kn = static_cast<const Act *>(a.k_new), *vn = static_cast<const Act *>(a.v_new);
  // (whole warps: the rows' threads shuffle)
  for (int64_t base = 0; base < end; base += kThreads) {
    const int64_t i = base + tid;
    const bool in = i < end;
    const int l_in = in ? static_cast<int>(div_nn(i, per_layer)) : 0;
    const int l = l0 + l_in, r = in ? static_cast<int>(i - static_cast<int64_t>(l_in) * per_layer) : 0;
    const int c = r % kPer, th = r / kPer, t = th / H, h = th - t * H;
    const int32_t slot = slots[t];
    const bool on = in && slot >= 0;
    float k0[N], k1[N], v0[N], v1[N];
    if (on) {
      const int64_t from = ((static_cast<int64_t>(l) * a.n_tokens + t0 + t) * H + h) * D + c * N;
      const uint4 a0 = __ldcs(reinterpret_cast<const uint4 *>(kn + from));
      const uint4 a1 = __ldcs(reinterpret_cast<const uint4 *>(kn + from + D / 2));
      const uint4 b0 = __ldcs(reinterpret_cast<const uint4 *>(vn + from));
      const uint4 b1 = __ldcs(reinterpret_cast<const uint4 *>(vn + from + D / 2));
      float x0[N], x1[N];
      Vec<Act>::unpack(a0, x0);
      Vec<Act>::unpack(a1, x1);
      Vec<Act>::unpack(b0, v0);
      Vec<Act>::unpack(b1, v1);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float2 cs = turn[t][c * N + j];
        if constexpr (kFp4) {
          fp4_turn(x0[j], x1[j], cs.x, cs.y, k0[j], k1[j]);
        } else {  // as the appends of the decode calls
          k0[j] = __fmaf_rn(x0[j], cs.x, -__fmul_rn(x1[j], cs.y));
          k1[j] = __fmaf_rn(x1[j], cs.x, __fmul_rn(x0[j], cs.y));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) k0[j] = k1[j] = v0[j] = v1[j] = 0.f;
    }
    const int64_t row = (static_cast<int64_t>(l) * H + h) * a.capacity + (on ? slot : 0);
    if constexpr (kFp4) {
      uint32_t kl, kh, vl, vh;
      const float ks = fp4_row(k0, k1, kl, kh);
      const float vs = fp4_row(v0, v1, vl, vh);
      if (on) {
        uint32_t *kd = reinterpret_cast<uint32_t *>(a.k_cache) + row * (D / 8);
        uint32_t *vd = reinterpret_cast<uint32_t *>(a.v_cache) + row * (D / 8);
        kd[c] = kl;
        kd[D / 16 + c] = kh;
        vd[c] = vl;
        vd[D / 16 + c] = vh;
        if (c == 0) static_cast<uint32_t *>(a.kv_scale)[row] = fp4_scale_word(ks, vs);
      }
    } else if (on) {
      Store *kd = static_cast<Store *>(a.k_cache) + row * D + c * N;
      Store *vd = static_cast<Store *>(a.v_cache) + row * D + c * N;
      if constexpr (sizeof(Store) == 1) {  // E4M3
        const float ki = 1.f / __ldg(a.k_scale + l * H + h), vi = 1.f / __ldg(a.v_scale + l * H + h);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          k0[j] *= ki;
          k1[j] *= ki;
          v0[j] *= vi;
          v1[j] *= vi;
        }
        *reinterpret_cast<uint2 *>(kd) = make_uint2(e4m3x4(k0), e4m3x4(k0 + 4));
        *reinterpret_cast<uint2 *>(kd + D / 2) = make_uint2(e4m3x4(k1), e4m3x4(k1 + 4));
        *reinterpret_cast<uint2 *>(vd) = make_uint2(e4m3x4(v0), e4m3x4(v0 + 4));
        *reinterpret_cast<uint2 *>(vd + D / 2) = make_uint2(e4m3x4(v1), e4m3x4(v1 + 4));
      } else {
        *reinterpret_cast<uint4 *>(kd) = Vec<Act>::pack(k0);
        *reinterpret_cast<uint4 *>(kd + D / 2) = Vec<Act>::pack(k1);
        *reinterpret_cast<uint4 *>(vd) = Vec<Act>::pack(v0);
        *reinterpret_cast<uint4 *>(vd + D / 2) = Vec<Act>::pack(v1);
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

// Grid row c (blockIdx.y) commits range c; its CTAs stride over the range's
// (layer, kv head, token) rows, 8 threads each.
__global__ void __launch_bounds__(kThreads) commit_fp4_kernel(const __grid_constant__ CommitArgs a,
                                                              const CommitScales scales) {
  __shared__ float cs[64], sn[64];
  const int c = blockIdx.y;
  const int n_tokens = a.n_tokens[c];
  const int64_t delta = a.delta[c];
  if (threadIdx.x < 64) rope_cos_sin_exact(delta, a.phase[threadIdx.x], &cs[threadIdx.x], &sn[threadIdx.x]);
  __syncthreads();
  const int64_t end = static_cast<int64_t>(a.n_layers) * a.n_kv_heads * n_tokens * 8;
  const uint32_t *ksrc = static_cast<const uint32_t *>(a.k_src);
  const uint2 *vsrc = static_cast<const uint2 *>(a.v_src);
  uint32_t *kdst = static_cast<uint32_t *>(a.k_dst);
  uint2 *vdst = static_cast<uint2 *>(a.v_dst);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  // (whole warps: the rows' threads shuffle)
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads; base < end; base += step) {
    const int64_t i = base + threadIdx.x;
    const bool on = i < end;
    const int ch = static_cast<int>(i & 7);
    const int64_t row = on ? i >> 3 : 0;
    const int64_t lh = div_nn(row, n_tokens), j = row - lh * n_tokens;
    const int64_t so = lh * a.src_capacity + a.src_begin[c] + j;
    const int64_t to = lh * a.dst_capacity + a.dst_offset[c] + j;
    uint32_t kl = 0, kh = 0, sw = 0;
    uint2 v = make_uint2(0, 0);
    if (on) {
      kl = __ldcs(ksrc + so * 16 + ch);
      kh = __ldcs(ksrc + so * 16 + 8 + ch);
      v = __ldcs(vsrc + so * 8 + ch);
      sw = __ldg(scales.src + so);
    }
    if (delta != 0) {  // (the same for the whole CTA)
      const float s = fp4_k_scale(sw);
      float x0[8], x1[8], y0[8], y1[8];
      fp4_levels8(kl, x0);
      fp4_levels8(kh, x1);
#pragma unroll
      for (int e = 0; e < 8; ++e) fp4_turn(x0[e] * s, x1[e] * s, cs[ch * 8 + e], sn[ch * 8 + e], y0[e], y1[e]);
      const float t = fp4_row(y0, y1, kl, kh);
      sw = fp4_scale_word(t, fp4_v_scale(sw));
    }
    if (on) {
      kdst[to * 16 + ch] = kl;
      kdst[to * 16 + 8 + ch] = kh;
      vdst[to * 8 + ch] = v;
      if (ch == 0) scales.dst[to] = sw;
    }
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
  int64_t work = 0;
  for (int c = 0; c < a.n_commits; ++c)
    work += static_cast<int64_t>(a.n_layers) * a.n_kv_heads * a.n_tokens[c] * 8;
  if (work == 0) return cudaSuccess;
  // about eight CTAs per SM in all, shared evenly by the commits
  int64_t ctas = (work + kThreads - 1) / kThreads;
  const int64_t cap = 8ll * sm_count();
  if (ctas > cap) ctas = cap;
  const int64_t per = (ctas + a.n_commits - 1) / a.n_commits;
  commit_fp4_kernel<<<dim3(static_cast<unsigned>(per), static_cast<unsigned>(a.n_commits)), kThreads, 0, s>>>(a, scales);
  return cudaGetLastError();
}

}  // namespace hw
