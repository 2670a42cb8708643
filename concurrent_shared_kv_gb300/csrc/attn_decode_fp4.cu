// attn_decode_fp4.cu - concurrent decode attention for 4-bit caches (E2M1 codes, a
// scale a token and kv head; head_dim 128) on the sm_100 tensor cores.
//
// The plan, the split over the CTAs, the records and the merge are those of the other
// caches (hw_device.cuh, hw_decode_plan.cuh), and so are the two products of a tile:
//   S^T [128 tokens x 32 columns] = K codes . Q~^T
//   O^T [128 d x 32 columns]     += V codes^T . P^T
// A tile is 16.5 KB here, a quarter of bf16's: DRAM brings one to an SM every 0.38 us,
// so what the other kernels hide behind their loads (1.2 us a tile with E4M3
// caches, the softmax of four warps) is what bounds this one.  It is built for it:
//
//  - Codes go from memory into the products.  The copy engine spreads 16 codes over 16
//    bytes (8 bytes of codes, 8 left), which is how kind::f8f6f4 reads 4-bit operands;
//    nothing is widened by a thread.  Both products are E2M1 x E4M3.
//  - Scales stay out of the products.  A token is a row of S^T, so its thread has the
//    one factor of its scores, and takes the value's scale into the weight:
//    w = 2^(s ks + log2 vs - m), O = sum w c, l = sum w / vs.  Two fused
//    multiply-adds an element, the ones that the sum and the shift cost anyway.  Scales
//    span 2^200, more than w's exponents: where a warp has a scale below 2^-8, l takes
//    2^(s ks - m) by itself, and a record's m is that of the scores alone.
//  - Sixteen softmax warps in two streams, one for even tiles, one for odd ones, with
//    scores, weights, maxima and outputs of their own: one stream's latencies (TMEM,
//    votes, fences) run under the other's arithmetic.  In a stream two threads share a
//    token, each with half the columns; columns go to the halves by turns, and
//    groups of four that hold none are skipped, so 20 columns cost 24, not 32.
//  - Q~ is held as kQParts E4M3 parts x = a + b/16 + ..., each the rounded remainder of those
//    before it (12 bits of every element; 2^-19 of the largest one where E4M3 runs out
//    of exponents), side by side on N (96 columns), and summed where S is read.  P is two
//    E4M3 parts side by side (N = 64), summed where records are written.  On N because an
//    instruction takes 32 + N / 4 clocks: a second part costs a quarter of a second one on K.
//  - A warp issues either product, and the scores of kLead tiles are ahead of the weights; K
//    and V share one ring, filled in the order of their use by one thread.
//
// Measured (40/8 heads, 4 rows): 262,144 tokens 79 us, 3.5 TB/s, 0.53 us a tile and SM, of which the chain
// product - TMEM - vote - exponentials - product is what two streams leave; 16,384 tokens
// 15.8 us a layer in a chain of layers (bf16 19.1, E4M3 21.4), of which 12 are trips to L2 at both
// ends.  (All columns a thread in eight warps: 92 us where two threads a token were 86; three
// streams 100; two tiles at a time in a stream 98 and more.)
//
// Warps: 0-7 softmax of stream 0 (0-3 the first half of the columns, 4-7 the other),
// 8-15 of stream 1, 16 TMA producer, 17 issues Q~ K, 18 P V, 19 rotated queries of
// segments behind the first, arrivals, appended tokens (the softmax warps do the first
// segment's queries: nothing can start before them).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cfloat>

#include "hw_decode_plan.cuh"
#include "hw_fp4.cuh"
#include "hw_rope_exact.cuh"

namespace hw {

namespace {

constexpr int kThreads = 640;
constexpr int kWarpTma = 16, kWarpQk = 17, kWarpPv = 18, kWarpQ = 19;
constexpr int kSoftWarps = 16;
constexpr uint32_t kTile = 128 * 128;      // a K or V tile in shared memory, 128-byte swizzled
constexpr uint32_t kTileTx = 128 * 64;     // the bytes of it that come from memory
constexpr int kSlots = 9;                  // of the ring
constexpr int kLead = 2;                   // tiles whose scores are asked for before the first one's weights
constexpr int kQParts = 3;
constexpr uint32_t kQPart = kN * 128;      // a part of Q~: [32 columns][128], 128-byte swizzled
constexpr uint32_t kQBytes = kQParts * kQPart;
constexpr uint32_t kPBytes = 128 * 64;     // P: [128 tokens][32 first parts, 32 second ones], 64-byte swizzled
constexpr int kHalf = kN / 2;              // columns of a softmax thread
// Weights are kept 2^kLift times larger than the running maximum asks for, and O is
// rescaled once one would pass 2^(kLift + kLazy) = 256 (E4M3 ends at 448): weights down to
// 2^-10 of the maximum keep both parts' precision (and smaller ones their sum: split_weights).
// The factor is in the record's m.  (2^5 and 2^3: 16K tokens 18.9 us where this is 17.9, chunks
// over 32K 25.8 for 24.2; 2^6 and 2^2: 19.8 and 27.6: references move more often.)
constexpr float kLift = 4.f, kLazy = 4.f;
// TMEM columns: S of either stream, its parts side by side, then O of (segment parity,
// stream): 32 columns for each part of P
constexpr uint32_t kSCols = kQParts * kN, kTmemO = 2 * kSCols, kTmemCols = 512;
static_assert(kTmemO + 4 * 2 * kN <= kTmemCols, "TMEM columns");

struct Fp4Smem {
  alignas(1024) uint8_t ring[kSlots][kTile];
  alignas(1024) uint8_t q[2][kQBytes];  // by segment parity
  alignas(1024) uint8_t p[2][2][kPBytes];  // by stream and buffer
  PlanShared ps;
  CtaPlan cp;
  PlanHeader hdr;
  // stream, half, parity of the stream's tile: the column maxima of the four warps
  alignas(16) float red[2][2][2][kHalf][4];
  alignas(16) float neg_ref[kSoftWarps][kHalf];  // a warp's own copy: minus its columns' references
  float hm[2][2][kN];          // segment parity, stream: reference maxima of the columns
  float hl[2][2][4][kN];       // and the warps' sums of weights
  int32_t nref[2];             // segment parity: references,
  float q_mul[2];              // the power of two that scores are to be multiplied with
  float qmax[kSoftWarps];
  int32_t abort_flag, plan_ok;
  uint32_t tmem_base;
  // what a softmax warp needs only between segments: its place in the units, the
  // segment whose records are due (registers are few in its loop over tiles)
  UnitPos walk[kSoftWarps];
  struct Due {
    int64_t sid;
    int32_t nq, cnt, first;
  } due[kSoftWarps];
  alignas(8) uint64_t kv_full[kSlots];
  uint64_t kv_empty[kSlots];
  uint64_t s_full[2], s_empty[2], p_full[2][2], p_empty[2][2];        // by stream (and buffer)
  uint64_t q_full[2], q_empty[2], o_full[2], o_empty[2], hand[2];     // by segment parity
  uint64_t rec_ready[4];                                              // by segment mod 4
  uint64_t plan_bar, app_bar, mma_done[2];
};
static_assert(sizeof(Fp4Smem) + 1024 <= 232448, "shared memory of one CTA per SM");
static_assert(sizeof(PlanHeader) % 16 == 0 && offsetof(Fp4Smem, hdr) % 16 == 0, "bulk copies");
static_assert(sizeof(MergeSmem<8>) <= kSlots * kTile, "merge scratch fits the ring");

// kind::f8f6f4, A E2M1 (format 5), B E4M3, fp32 accumulator.
constexpr uint32_t idesc_fp4(int M, int N, int a_mn, int b_mn) { return idesc_e4m3(M, N, a_mn, b_mn) | (5u << 7); }

__device__ __forceinline__ void set_abort(Fp4Smem &S, const DecodeArgs &a) {
  if (atomicExch(&S.abort_flag, 1) == 0) flag_error(a.err, HW_DEV_TIMEOUT);
}
__device__ __forceinline__ bool aborted(Fp4Smem &S) { return *reinterpret_cast<volatile int32_t *>(&S.abort_flag) != 0; }
// Bounded wait, suspended; on a timeout the CTA winds down (no wait blocks any more
// and every role runs to its end).
__device__ __forceinline__ void idle_wait(Fp4Smem &S, const DecodeArgs &a, uint64_t *bar, uint32_t parity) {
  if (!mbar_try(bar, parity)) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
      if (aborted(S)) break;
      if (clock64() - t0 > kWaitLimit) {
        set_abort(S, a);
        break;
      }
    }
  }
  __syncwarp();
}
// idle_wait by some lanes of a warp.
__device__ __forceinline__ void idle_wait_lane(Fp4Smem &S, const DecodeArgs &a, uint64_t *bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (aborted(S)) break;
    if (clock64() - t0 > kWaitLimit) {
      set_abort(S, a);
      break;
    }
  }
}
// The same spinning, with one answer for the warp.
__device__ __forceinline__ bool warp_spin(Fp4Smem &S, const DecodeArgs &a, uint64_t *bar, uint32_t parity) {
  bool ok = mbar_test(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    while (!(ok = mbar_test(bar, parity))) {
      if (aborted(S)) break;
      if (clock64() - t0 > kWaitLimit) {
        set_abort(S, a);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// A place in the ring.
struct RingPos {
  int s;
  uint32_t phase;
  __device__ __forceinline__ void next() {
    if (++s == kSlots) {
      s = 0;
      phase ^= 1;
    }
  }
};

// Column qi's place among S's columns: by turns in the two halves.
__device__ __forceinline__ int column_place(int qi) { return (qi & 1) * kHalf + (qi >> 1); }

// ------------------------------------------------------------------ producer

// One thread, which has under 800 clocks for a tile's two copies: within a segment a
// tile's place is the one before it plus 128 tokens, and a V's is that of the K kLead
// tiles before.  Tiles are loaded in the order of their use, K(0) .. K(kLead-1), V(0),
// K(kLead), V(1), ...: step j takes V(j - kLead), then K(j).
struct Producer {
  RingPos at;
  int count;  // copies issued so far
  int step;
  int row[kLead + 1], h[kLead + 1];  // the K's of this step and those before it
  UnitPos x;  // the segment's first unit of the CTA's
  int left;   // tiles of the segment from this one on
};

__device__ __forceinline__ void start(const DecodeArgs &a, const Fp4Smem &S, Producer &p) {
  p.at = {0, 0};
  p.count = p.step = 0;
  p.x = unit_pos(S.ps.plan, a.n_blocks, S.cp.u0);
  p.left = p.x.tiles - p.x.t;
#pragma unroll
  for (int k = 0; k <= kLead; ++k) p.row[k] = p.h[k] = 0;
  p.row[0] = S.ps.plan.start[p.x.b] + p.x.t * kT;
  p.h[0] = p.x.h;
}

// Steps up to j1 of n tiles, while `room` copies are left; app_tile: the first tile with
// a new token (or -1), loaded once the tokens are written (and fenced for the copy engine).
__device__ __forceinline__ void produce(const DecodeArgs &a, Fp4Smem &S, const CUtensorMap *tk, const CUtensorMap *tv,
                                        Producer &p, int n, int j1, int room, int app_tile) {
  const uint64_t pol = policy_evict_first();
  const PlanCore &P = S.ps.plan;
  auto spin = [&](uint64_t *bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_test(bar, parity)) {
      if (aborted(S)) return false;
      if (clock64() - t0 > kWaitLimit) {
        set_abort(S, a);
        return false;
      }
    }
    return true;
  };
  auto load = [&](const CUtensorMap *m, int row, int h) {
    if (p.count >= kSlots && !spin(&S.kv_empty[p.at.s], p.at.phase ^ 1)) return false;
    mbar_arrive_expect_tx(&S.kv_full[p.at.s], kTileTx);
    tma_load_3d(S.ring[p.at.s], m, &S.kv_full[p.at.s], 0, row, h, pol);
    ++p.count;
    p.at.next();
    return true;
  };
  for (; p.step < j1 && p.count + 2 <= room; ++p.step) {
    const int j = p.step;
    if (j >= kLead && !load(tv, p.row[kLead], p.h[kLead])) return;
    if (j < n) {
      if (j == app_tile && !spin(&S.app_bar, 0)) return;
      // the tile's scales into L2 (its threads load them shortly before they need them);
      // of a tile that the block fills, whole 16-byte pieces
      if (p.left > 1)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                         (reinterpret_cast<uint64_t>(a.kv_scale + static_cast<int64_t>(p.h[0]) * a.capacity + p.row[0]) + 15) &
                         ~15ull),
                     "n"(kT * 4 - 16)
                     : "memory");
      if (!load(tk, p.row[0], p.h[0])) return;
    }
#pragma unroll
    for (int k = kLead; k > 0; --k) {
      p.row[k] = p.row[k - 1];
      p.h[k] = p.h[k - 1];
    }
    p.row[0] += kT;
    if (--p.left == 0) {
      p.x.t = p.x.tiles - 1;
      unit_pos_next(P, a.n_blocks, p.x);
      p.left = p.x.tiles - p.x.t;
      p.row[0] = P.start[p.x.b] + p.x.t * kT;
      p.h[0] = p.x.h;
    }
  }
}

// No copy may still be landing when the CTA retires.
__device__ void drain(Fp4Smem &S, const Producer &p) {
  RingPos back = p.count >= kSlots ? RingPos{p.at.s, p.at.phase ^ 1} : RingPos{0, 0};
  for (int j = min(p.count, kSlots); j > 0; --j, back.next()) mbar_wait(&S.kv_full[back.s], back.phase);
}

// --------------------------------------------------------------- MMA issuers
//
// A warp for either product: neither then waits for what the other one waits for, and the
// tensor cores have the one's instructions while the other looks at its barriers
// (about 60 clocks each).  An instruction of 32 bytes along K takes 32 + N / 4 clocks
// (measured, N from 32 to 128), so parts stand side by side on N, not one after the other
// on K: 4 x 56 clocks for S, 4 x 48 for O.

// Walks a CTA's tiles segment by segment.
struct SegWalk {
  UnitPos x;
  int seg, left;  // segment, tiles left of it
  __device__ __forceinline__ SegWalk(const DecodeArgs &a, const PlanCore &P, int64_t u0)
      : x(unit_pos(P, a.n_blocks, u0)), seg(-1), left(0) {}
  // On to tile i of n: whether it starts a segment.
  __device__ __forceinline__ bool next(const DecodeArgs &a, const PlanCore &P, int i, int n) {
    const bool first = left == 0;
    if (first) {
      if (seg >= 0) {
        x.t = x.tiles - 1;
        unit_pos_next(P, a.n_blocks, x);
      }
      ++seg;
      left = min(n - i, x.tiles - x.t);
    }
    --left;
    return first;
  }
};

__device__ void qk_issuer(const DecodeArgs &a, Fp4Smem &S, uint32_t tmem, int64_t u0, int n) {
  constexpr uint32_t idesc = idesc_fp4(128, kSCols, 0, 0);
  const uint64_t k_desc = smem_desc(smem_u32(S.ring[0]), 16, 1024, kSw128);
  const uint64_t q_desc = smem_desc(smem_u32(S.q[0]), 16, 1024, kSw128);
  SegWalk w(a, S.ps.plan, u0);
  RingPos at = {0, 0};
  for (int i = 0; i < n; ++i) {
    const int st = i & 1;
    const bool first = w.next(a, S.ps.plan, i, n);
    if (first && !warp_spin(S, a, &S.q_full[w.seg & 1], (w.seg >> 1) & 1)) return;
    if (!warp_spin(S, a, &S.s_empty[st], ((i >> 1) & 1) ^ 1)) return;
    if (!warp_spin(S, a, &S.kv_full[at.s], at.phase)) return;
    tc_fence_after();
    if (elect_one()) {
      const uint64_t k0 = k_desc + ((at.s * kTile) >> 4), q = q_desc + (((w.seg & 1) * kQBytes) >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k)  // 4 steps of 32 elements
        mma_f8(tmem + st * kSCols, k0 + ((k * 32) >> 4), q + ((k * 32) >> 4), idesc, k > 0);
      mma_commit(&S.s_full[st]);
      mma_commit(&S.kv_empty[at.s]);
      if (w.left == 0) mma_commit(&S.q_empty[w.seg & 1]);
    }
    __syncwarp();
    // (the next K: behind the next V from the kLead-th on)
    at.next();
    if (i + 1 >= kLead) at.next();
  }
}

__device__ void pv_issuer(const DecodeArgs &a, Fp4Smem &S, uint32_t tmem, int64_t u0, int n) {
  constexpr uint32_t idesc = idesc_fp4(128, 2 * kN, 1, 1);
  const uint64_t v_desc = smem_desc(smem_u32(S.ring[0]), kTile, 1024, kSw128);
  const uint64_t p_desc = smem_desc(smem_u32(S.p[0][0]), 512, 512, kSw64);
  SegWalk w(a, S.ps.plan, u0);
  RingPos at = {0, 0};
  for (int k = min(kLead, n); k > 0; --k) at.next();  // V(0) is behind the first K's
  int in = 0;  // the tile's index in its segment
  for (int i = 0; i < n; ++i) {
    const int st = i & 1, buf = (i >> 1) & 1;
    if (w.next(a, S.ps.plan, i, n)) {
      in = 0;
      if (!warp_spin(S, a, &S.o_empty[w.seg & 1], ((w.seg >> 1) & 1) ^ 1)) return;
    }
    if (!warp_spin(S, a, &S.kv_full[at.s], at.phase)) return;
    if (!warp_spin(S, a, &S.p_full[st][buf], (i >> 2) & 1)) return;
    tc_fence_after();
    const bool first = in < 2;  // of its stream in this segment
    ++in;
    if (elect_one()) {
      const uint32_t o = tmem + kTmemO + ((w.seg & 1) * 2 + st) * 2 * kN;
      const uint64_t v = v_desc + ((at.s * kTile) >> 4), p = p_desc + (((st * 2 + buf) * kPBytes) >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k)  // 4 steps of 32 tokens
        mma_f8(o, v + ((k * 4096) >> 4), p + ((k * 2048) >> 4), idesc, !(first && k == 0));
      mma_commit(&S.p_empty[st][buf]);
      mma_commit(&S.kv_empty[at.s]);
      if (w.left == 0) mma_commit(&S.o_full[w.seg & 1]);
    }
    __syncwarp();
    at.next();
    if (i + kLead < n) at.next();  // (the K between this V and the next)
  }
}

// ------------------------------------------------------------------- queries

__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// A column's largest pair length over the item's elements, squared: turned
// elements are no longer than that.  One that is not finite makes its own column NaN, and
// no other: it does not count for the exponent that the segment's columns share.
__device__ __forceinline__ float item_reach(const QItem &it) {
  const uint32_t lo[4] = {it.lo.x, it.lo.y, it.lo.z, it.lo.w}, hi[4] = {it.hi.x, it.hi.y, it.hi.z, it.hi.w};
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a0 = __uint_as_float(lo[e] << 16), a1 = __uint_as_float(hi[e] << 16);
    const float b0 = __uint_as_float(lo[e] & 0xffff0000u), b1 = __uint_as_float(hi[e] & 0xffff0000u);
    m = max_nan(m, max_nan(__fmaf_rn(a0, a0, a1 * a1), __fmaf_rn(b0, b0, b1 * b1)));
  }
  return m;
}
// The exponent e with |y| < 2^(e + 8) (E4M3 ends at 448) for a segment whose squared pair
// lengths reach `reach` before scale * log2(e); and 2^e.
__device__ __forceinline__ int part_exponent(const DecodeArgs &a, float reach) {
  const float r = reach * a.scale_log2 * a.scale_log2;
  return max(-120, min(((static_cast<int>(__float_as_uint(r) >> 23) - 127) >> 1) - 7, 120));
}
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// Two E4M3 codes (low byte first) as two fp32, exactly.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3));
  return __half22float2(h);
}

// cos and sin of the angle rel * phase, from its upper 32 bits (2^-32 turns are far
// below what the parts keep) by the fast hardware functions.
__device__ __forceinline__ void turn_of(int64_t rel, uint64_t phase, float *c, float *s) {
  const int32_t turns = static_cast<int32_t>((static_cast<uint64_t>(rel) * phase) >> 32);
  __sincosf(static_cast<float>(turns) * (3.14159265358979323846f * 0x1p-31f), s, c);
}
// cos and sin of an item's 8 elements.
__device__ __forceinline__ void item_turns(const Fp4Smem &S, int64_t rel, int c, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) turn_of(rel, S.ps.cache.phase[8 * c + e], &cs[e], &sn[e]);
}

// (x, y) as kQParts E4M3 parts, each the remainder of those before it times 16.
__device__ __forceinline__ void split_query(float2 y, uint32_t (&q)[kQParts]) {
#pragma unroll
  for (int j = 0; j < kQParts; ++j) {
    q[j] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    if (j + 1 < kQParts) {
      const float2 v = e4m3x2_values(q[j]);
      y = make_float2((y.x - v.x) * 16.f, (y.y - v.y) * 16.f);
    }
  }
}

// The item turned, scaled by mul and split into parts, each the remainder of those before
// it times 16, into row `place` of Q~'s parts: 8 codes at byte 8c, 8 at 64 + 8c, 16-byte
// chunks swizzled.
__device__ __forceinline__ void store_item(const QItem &it, const float (&cs)[8], const float (&sn)[8], uint32_t qbase,
                                           int place, int c, float mul) {
  const uint32_t lo32[4] = {it.lo.x, it.lo.y, it.lo.z, it.lo.w}, hi32[4] = {it.hi.x, it.hi.y, it.hi.z, it.hi.w};
  uint32_t w[kQParts][4];
#pragma unroll
  for (int j = 0; j < kQParts; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) w[j][k] = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 y0, y1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x0 = __uint_as_float(h ? (lo32[e] & 0xffff0000u) : (lo32[e] << 16));
      const float x1 = __uint_as_float(h ? (hi32[e] & 0xffff0000u) : (hi32[e] << 16));
      (h ? y0.y : y0.x) = (x0 * cs[2 * e + h] - x1 * sn[2 * e + h]) * mul;
      (h ? y1.y : y1.x) = (x1 * cs[2 * e + h] + x0 * sn[2 * e + h]) * mul;
    }
    uint32_t q0[kQParts], q1[kQParts];
    split_query(y0, q0);
    split_query(y1, q1);
#pragma unroll
    for (int j = 0; j < kQParts; ++j) {
      w[j][e >> 1] |= q0[j] << (16 * (e & 1));
      w[j][2 + (e >> 1)] |= q1[j] << (16 * (e & 1));
    }
  }
  const uint32_t row = qbase + place * 128, sub = 8u * (c & 1);
  const uint32_t c0 = ((static_cast<uint32_t>(c >> 1) ^ (place & 7)) << 4) + sub;
  const uint32_t c1 = ((static_cast<uint32_t>(4 + (c >> 1)) ^ (place & 7)) << 4) + sub;
#pragma unroll
  for (int j = 0; j < kQParts; ++j) {
    st_shared_v2(row + j * kQPart + c0, w[j][0], w[j][1]);
    st_shared_v2(row + j * kQPart + c1, w[j][2], w[j][3]);
  }
}

// Segment 0's queries, by the softmax warps (nothing else can start before them): a
// thread has 4 elements of the first half of a column's, and the 4 that they turn with.
__device__ void query_prologue(const DecodeArgs &a, Fp4Smem &S) {
  static_assert(kSoftWarps == kN / 2, "16 threads a column");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, qi = t >> 4, c = t & 15;
  NamedSync<5, 32 * kSoftWarps> sync;
  const SegQ &X = S.cp.pre[0];
  const bool on = qi < min(X.m.n_ref * (a.n_q_heads / a.n_kv_heads), kN);
  uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
  int64_t rel = 0;
  if (on) {
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + static_cast<int64_t>(X.qrow[qi]) * 128 + 4 * c;
    lo = __ldg(reinterpret_cast<const uint2 *>(qp));
    hi = __ldg(reinterpret_cast<const uint2 *>(qp + 64));
    rel = X.rel[qi];
  }
  float cs[4], sn[4];  // (while the loads are under way)
#pragma unroll
  for (int e = 0; e < 4; ++e) turn_of(rel, S.ps.cache.phase[4 * c + e], &cs[e], &sn[e]);
  float x0[4], x1[4], reach = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t l = e < 2 ? lo.x : lo.y, h = e < 2 ? hi.x : hi.y;
    x0[e] = __uint_as_float(e & 1 ? l & 0xffff0000u : l << 16);
    x1[e] = __uint_as_float(e & 1 ? h & 0xffff0000u : h << 16);
    reach = max_nan(reach, __fmaf_rn(x0[e], x0[e], x1[e] * x1[e]));
  }
  const bool finite = reach < INFINITY;
  reach = warp_max(finite ? reach : 0.f);
  if (lane == 0) S.qmax[warp] = reach;
  sync();
  reach = warp_max(S.qmax[lane & (kSoftWarps - 1)]);
  const int ex = part_exponent(a, reach);
  if (on) {
    const float mul = finite ? a.scale_log2 * two_to(-ex) : NAN;
    uint32_t w0[kQParts], w1[kQParts];
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      uint32_t q0[kQParts], q1[kQParts];
      split_query(make_float2((x0[e] * cs[e] - x1[e] * sn[e]) * mul, (x0[e + 1] * cs[e + 1] - x1[e + 1] * sn[e + 1]) * mul), q0);
      split_query(make_float2((x1[e] * cs[e] + x0[e] * sn[e]) * mul, (x1[e + 1] * cs[e + 1] + x0[e + 1] * sn[e + 1]) * mul), q1);
#pragma unroll
      for (int j = 0; j < kQParts; ++j) {
        w0[j] = e ? w0[j] | q0[j] << 16 : q0[j];
        w1[j] = e ? w1[j] | q1[j] << 16 : q1[j];
      }
    }
    // (codes at byte 4c and 64 + 4c of the row, 16-byte chunks swizzled)
    const int place = column_place(qi);
    const uint32_t row = smem_u32(S.q[0]) + place * 128 + 4 * (c & 3);
    const uint32_t c0 = (c >> 2 ^ (place & 7)) << 4, c1 = ((4 + (c >> 2)) ^ (place & 7)) << 4;
#pragma unroll
    for (int j = 0; j < kQParts; ++j) {
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + j * kQPart + c0), "r"(w0[j]) : "memory");
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + j * kQPart + c1), "r"(w1[j]) : "memory");
    }
  }
  if (t == 0) {
    S.nref[0] = X.m.n_ref;
    S.q_mul[0] = two_to(ex);
  }
  fence_proxy_async_smem();
  sync();
  if (t == 0) mbar_arrive(&S.q_full[0]);
}

// Queries of segments 1, 2, ..., and the arrivals of finished ones two segments
// late, by warp 19 (as in the other tensor-core kernel).
template <bool kLimit>
__device__ void qprep(const DecodeArgs &a, Fp4Smem &S, int64_t u1) {
  const int lane = threadIdx.x & 31;
  const int G = a.n_q_heads / a.n_kv_heads;
  auto arrivals = [&](int done) {
    idle_wait(S, a, &S.rec_ready[done & 3], (done >> 2) & 1);
    arrive_segment(a, S.cp.pre[done % kPre].m, lane);
  };
  int64_t u = S.cp.us[1];
  int64_t u_prep = S.cp.us[kPre - 1] < u1 ? next_segment(S.ps.plan, a.n_blocks, S.cp.us[kPre - 1]) : u1;
  for (int seg = 1;; ++seg) {
    if (u >= u1) {
      if (seg >= 2) arrivals(seg - 2);
      arrivals(seg - 1);
      break;
    }
    const SegQ &X = S.cp.pre[seg % kPre];
    const int n_ref = X.m.n_ref, par = seg & 1;
    // a lane's items: (reference, chunk), for each its q heads, which share a turn (32 in all
    // at most: 32 of one reference's)
    float reach = 0.f;
    uint32_t bad = 0;  // those that are not finite
    int k = 0;
    for (int it = lane; it < n_ref * 8; it += 32)
      for (int g = 0; g < G; ++g) {
        QItem raw;
        load_item(a, X, (it >> 3) * G + g, it & 7, raw);
        const float r = item_reach(raw);
        const bool finite = r < INFINITY;
        reach = fmaxf(reach, finite ? r : 0.f);
        bad |= (finite ? 0u : 1u) << k++;
      }
    k = 0;
    const int e = part_exponent(a, warp_max_nonneg(reach));
    const float mul = a.scale_log2 * two_to(-e);
    if (seg >= 2) idle_wait(S, a, &S.q_empty[par], ((seg >> 1) - 1) & 1);
    if (lane == 0) {
      S.nref[par] = n_ref;
      S.q_mul[par] = two_to(e);
    }
    for (int it = lane; it < n_ref * 8; it += 32) {
      float cs[8], sn[8];
      item_turns(S, X.rel[(it >> 3) * G], it & 7, cs, sn);
      for (int g = 0; g < G; ++g) {
        const int qi = (it >> 3) * G + g;
        QItem raw;
        load_item(a, X, qi, it & 7, raw);
        store_item(raw, cs, sn, smem_u32(S.q[par]), column_place(qi), it & 7, bad >> k++ & 1 ? NAN : mul);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_full[par]);
    if (seg >= 2) {
      arrivals(seg - 2);
      __syncwarp();  // the slot of segment seg - 2 is read; it now takes segment seg + 2
      if (u_prep < u1) {
        const UnitPos x = unit_pos(S.ps.plan, a.n_blocks, u_prep);
        seg_pre<kLimit>(a, S.ps.plan, S.ps.cache, S.cp.pre[(seg + 2) % kPre], x.b, x.g, x.h, lane);
        u_prep = x.seg_first + x.tiles;
      }
      __syncwarp();
    }
    u = next_segment(S.ps.plan, a.n_blocks, u);
  }
}

// The CTA's new tokens (hw_attn_append_decode_planned_fp4), by warp 19, a (row, kv head) pair
// at a time, lane l the elements 2l, 2l + 1 and those that they turn with: the bits that
// hw_cache_write stores.  (With 8 lanes a pair it took 7 us, one warp's chain of
// 1500 instructions, and everything behind the first new token waits for it.)
__device__ void append_tokens(const DecodeArgs &a, Fp4Smem &S, int64_t u0, int64_t u1) {
  const int lane = threadIdx.x & 31;
  const PlanCore &P = S.ps.plan;
  const int Hkv = a.n_kv_heads, npairs = a.n_rows * Hkv;
  auto scale_of = [](float x0, float x1, float x2, float x3) {
    float top = max_nan(max_nan(fabsf(x0), fabsf(x1)), max_nan(fabsf(x2), fabsf(x3)));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    return fp4_scale(top);
  };
  auto write = [&](int pr, int pos, int row) {
    const uint32_t *kn = static_cast<const uint32_t *>(a.k_new) + static_cast<int64_t>(pr) * 64 + lane;
    const uint32_t *vn = static_cast<const uint32_t *>(a.v_new) + static_cast<int64_t>(pr) * 64 + lane;
    const uint32_t k0 = __ldg(kn), k1 = __ldg(kn + 32), v0 = __ldg(vn), v1 = __ldg(vn + 32);
    float cs[2], sn[2];  // (while the loads are under way)
#pragma unroll
    for (int j = 0; j < 2; ++j) rope_cos_sin_exact(pos, S.ps.cache.phase[2 * lane + j], &cs[j], &sn[j]);
    float y[4];
    fp4_turn(__uint_as_float(k0 << 16), __uint_as_float(k1 << 16), cs[0], sn[0], y[0], y[2]);
    fp4_turn(__uint_as_float(k0 & 0xffff0000u), __uint_as_float(k1 & 0xffff0000u), cs[1], sn[1], y[1], y[3]);
    const float x[4] = {__uint_as_float(v0 << 16), __uint_as_float(v0 & 0xffff0000u), __uint_as_float(v1 << 16),
                        __uint_as_float(v1 & 0xffff0000u)};
    const float ks = scale_of(y[0], y[1], y[2], y[3]), vs = scale_of(x[0], x[1], x[2], x[3]);
    uint32_t c[4] = {0, 0, 0, 0};
    if (ks > 0.f) {
      c[0] = fp4_encode2(y[0], y[1], ks);
      c[1] = fp4_encode2(y[2], y[3], ks);
    }
    if (vs > 0.f) {
      c[2] = fp4_encode2_bf16(x[0], x[1], vs);
      c[3] = fp4_encode2_bf16(x[2], x[3], vs);
    }
    const int64_t at = static_cast<int64_t>(pr % Hkv) * a.capacity + row;
    uint8_t *kc = static_cast<uint8_t *>(const_cast<void *>(a.k)) + at * 64, *vc = static_cast<uint8_t *>(const_cast<void *>(a.v)) + at * 64;
    kc[lane] = static_cast<uint8_t>(c[0]);
    kc[32 + lane] = static_cast<uint8_t>(c[1]);
    vc[lane] = static_cast<uint8_t>(c[2]);
    vc[32 + lane] = static_cast<uint8_t>(c[3]);
    if (lane == 0) const_cast<uint32_t *>(a.kv_scale)[at] = fp4_scale_word(ks, vs);
  };
  if (S.cp.app_n <= kAppList) {
    for (int e = 0; e < S.cp.app_n; ++e) write(S.cp.app_pair[e], S.cp.app_pos[e], S.cp.app_row[e]);
  } else {
    // more than the plan lists: every pair is checked (each CTA that reads a token's
    // tile writes it, the same bytes, before its own copy of the tile)
    for (int base = 0; base < npairs; base += 32) {
      const int pr = base + lane;
      int pos = 0, row = 0;
      bool mine = false;
      if (pr < npairs) {
        const int r = pr / Hkv, h = pr - r * Hkv;
        const int b = __ldg(a.append_block + r);
        if (b >= 0 && b < a.n_blocks && P.tiles[b] > 0) {
          pos = __ldg(a.append_pos + r);
          if (pos >= 0 && pos < P.len[b]) {
            mine = tile_unit_in(P, b, h, pos / kT, u0, u1) >= 0;
            row = P.start[b] + pos;
          }
        }
      }
      for (unsigned m = __ballot_sync(0xffffffffu, mine); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        write(__shfl_sync(0xffffffffu, pr, src), __shfl_sync(0xffffffffu, pos, src), __shfl_sync(0xffffffffu, row, src));
      }
    }
  }
  __threadfence_block();
  asm volatile("fence.proxy.async.global;" ::: "memory");
  __syncwarp();
  if (lane == 0) mbar_arrive(&S.app_bar);
}

// ------------------------------------------------------------------- softmax

// Whether any of the 128 threads of barrier `id` says so.
__device__ __forceinline__ bool vote_128(int id, bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %2, 0;\n\t"
      "bar.red.or.pred po, %1, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out)
      : "r"(id), "r"(pred ? 1u : 0u)
      : "memory");
  return out != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float2 as_pair(uint32_t x, uint32_t y) {
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}

// Butterflies over the warp: on entry v[j] is this lane's value of column j, on exit
// v[0] is the whole warp's sum (largest one) of column lane & 15.
template <bool kMax>
__device__ __forceinline__ void join_columns(float (&v)[kHalf], int lane) {
#pragma unroll
  for (int off = kHalf / 2; off >= 1; off >>= 1) {
#pragma unroll
    for (int k = 0; k < off; ++k) {
      const bool up = (lane & off) != 0;
      const float mine = up ? v[k + off] : v[k];
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + off], off);
      v[k] = kMax ? fmaxf(mine, other) : mine + other;
    }
  }
  const float other = __shfl_xor_sync(0xffffffffu, v[0], 16);
  v[0] = kMax ? fmaxf(v[0], other) : v[0] + other;
}
__device__ __forceinline__ void sum_columns(float (&v)[kHalf], int lane) { join_columns<false>(v, lane); }
__device__ __forceinline__ void max_columns(float (&v)[kHalf], int lane) { join_columns<true>(v, lane); }

// x, y (at most 448) as two E4M3 parts each, x = hi + lo / 16: the codes of hi in the
// low half of the word, those of lo in the high one.  fp16 in between keeps 11 bits,
// more than the parts do together.  The remainder is taken from the code that is stored (E4M3's
// steps are 2^-9 below 2^-6), and lo's own rounding there is dithered: `dither` lies within half a
// step and is spread evenly over a segment's tokens, so that weights smaller than lo's step
// are there in the sum, however many of them stand below one large one.  (To nearest,
// 16,384 tokens at 2^-18 of the largest weight would be 6 % of the sum, and lost.  What
// is 0 stays 0, what is exact stays exact.)
__device__ __forceinline__ void split_weights(float x, float y, __half2 dither, uint16_t &hi, uint16_t &lo) {
  const __half2 v = __floats2half2_rn(x, y);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
  uint32_t top;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(top) : "h"(hi));
  const __half2 rest = __hfma2(__hsub2(v, *reinterpret_cast<const __half2 *>(&top)), __float2half2_rn(16.f), dither);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t *>(&rest)));
}
// The dither of a block's token: within 2^-10, golden steps from token to token.
__device__ __forceinline__ __half2 weight_dither(int token) {
  return __float2half2_rn(static_cast<float>(static_cast<int32_t>(token * 0x9e3779b9u)) * 0x1p-41f);
}

// l * 2^d, from half = 2^(d / 2): l is up to 2^100 times what O is (values of 2^-100), and 2^d
// alone may be below fp32's range.
__device__ __forceinline__ float l_shrink(float l, float half) { return l * half * half; }

// Records of a finished segment: every warp joins the two streams' outputs of 8 of its
// half's columns (stream 0's warps the first 8 places, stream 1's the others).  m has the
// values' scales in it and l has not, so a power of two is taken from O and l into m that leaves
// l between 1 and 2: then m is that of the scores, and the merge needs to know of no scales.
__device__ __noinline__ void segment_records(const DecodeArgs &a, Fp4Smem &S, uint32_t tmem, int seg) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int st = warp >> 3, half = (warp >> 2) & 1, qd = warp & 3, par = seg & 1;
  const uint32_t tl = tmem + (static_cast<uint32_t>(qd * 32) << 16) + kTmemO + par * 4 * kN;
  const int place = half * kHalf + st * 8;  // of the first column
  const Fp4Smem::Due due = S.due[warp];
  const int nq = due.nq;
  idle_wait(S, a, &S.hand[par], (seg >> 1) & 1);
  // lane (s, j): column j's sum and reference in stream s, joined, and the factor of that stream's O
  float m, l, f;
  {
    const int s = (lane >> 3) & 1, k = place + (lane & 7);
    const float mine = S.hm[par][s][k], other = S.hm[par][s ^ 1][k];
    const float *hl = &S.hl[par][s][0][k];
    m = fmaxf(mine, other);
    l = l_shrink(hl[0] + hl[kN] + hl[2 * kN] + hl[3 * kN], ex2(0.5f * (mine - m)));
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    const int e = l > 0.f && l < INFINITY ? (__float_as_int(l) >> 23) - 127 : 0;
    l = __int_as_float(__float_as_int(l) - (e << 23));
    f = ex2((mine - m) - static_cast<float>(e));
    m += static_cast<float>(e);
  }
  idle_wait(S, a, &S.o_full[par], (seg >> 1) & 1);
  tc_fence_after();
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = 0.f;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (due.cnt < 2 && s != due.first) continue;  // the stream had no tile of this segment
    uint32_t hi[8], lo[8];
    tmem_ld8(tl + s * 2 * kN + place, hi);
    tmem_ld8(tl + s * 2 * kN + kN + place, lo);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      o[j] = __fmaf_rn(__fmaf_rn(__uint_as_float(lo[j]), 0.0625f, __uint_as_float(hi[j])),
                       __shfl_sync(0xffffffffu, f, s * 8 + j), o[j]);
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&S.o_empty[par]);
  const int64_t slot = due.sid + S.cp.c_log;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int qi = 2 * (st * 8 + j) + half;
    if (qi < nq) record_ptr(a, slot, qi)[qd * 32 + lane] = o[j];
  }
  if (qd == 0 && lane < 8) {
    const int qi = 2 * (st * 8 + lane) + half;
    if (qi < nq) *reinterpret_cast<float2 *>(record_ptr(a, slot, qi) + 128) = make_float2(m, l);
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(&S.rec_ready[seg & 3]);
}

template <bool kAppend, bool kLimit>
__device__ void softmax_role(const DecodeArgs &a, Fp4Smem &S, uint32_t tmem, int64_t u0, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int st = warp >> 3, half = (warp >> 2) & 1, qd = warp & 3;
  const int row = qd * 32 + lane;  // token of the tile
  const int bar = 1 + st * 2 + half;
  const uint32_t tl = tmem + (static_cast<uint32_t>(qd * 32) << 16);
  const int G = a.n_q_heads / a.n_kv_heads;
  const PlanCore &P = S.ps.plan;
  const uint32_t pbase = smem_u32(S.p[st][0]) + row * 64, swz = (row >> 1) & 3;
  const uint32_t p_hi = pbase + ((half ^ swz) << 4), p_lo = pbase + (((2 + half) ^ swz) << 4);
  const int app_tile = kAppend && S.cp.app_n > 0 ? S.cp.app_tile : INT32_MAX;

  // A wait that gives up (HW_DEV_TIMEOUT) does not leave the loops: all threads keep
  // the same control flow, so the votes are always reached by all 128.
  // A column's reference is the exponent that its weights are taken against (its maximum
  // less kLift), the same in the four warps; ref_mine: column (lane & 15)'s, in shared memory
  // (negative) all of the half's, which would spill from registers.  Columns past the
  // segment's have inf there, and weights of 0.  One whose tokens are all masked keeps
  // -FLT_MAX (not -inf: its weights are then 2^-inf = 0).
  float l[kHalf], ref_mine;
  const float4 *neg_ref = reinterpret_cast<const float4 *>(S.neg_ref[warp]);
  int pend = -1;
  if (lane == 0) S.walk[warp] = unit_pos(P, a.n_blocks, u0);
  __syncwarp();
  for (int i0 = 0, seg = 0; i0 < n; ++seg) {
    const int par = seg & 1;
    int len, t0, i_end;  // the block's tokens; the first tile less i0; where the segment ends
    const uint32_t *scales;  // of this thread's token in tile 0
    {
      const UnitPos x = S.walk[warp];
      len = P.len[x.b];
      t0 = x.t - i0;
      i_end = i0 + min(n - i0, x.tiles - x.t);
      scales = a.kv_scale + static_cast<int64_t>(x.h) * a.capacity + P.start[x.b] + row;
    }
    // the scales of the stream's next tile, loaded a tile ahead (past the block: 1, and masked)
    auto scales_of = [&](int i) -> uint32_t {
      if (i >= i_end || (i + t0) * kT + row >= len) return 0x3f803f80u;
      if (kAppend && i >= app_tile) idle_wait_lane(S, a, &S.app_bar, 0);
      return __ldcg(scales + static_cast<int64_t>(i + t0) * kT);
    };
    int i = i0 + ((i0 ^ st) & 1);
    uint32_t sw_next = scales_of(i);
    idle_wait(S, a, &S.q_full[par], (seg >> 1) & 1);
    const int nq = min(S.nref[par] * G, kN);
    const int nh = (nq + 1 - half) >> 1;  // the half's columns
    const float q_mul = S.q_mul[par];
    int minlim = INT32_MAX, lim_mine = INT32_MAX;
    if constexpr (kLimit) {
      const SegQ &X = S.cp.pre[seg % kPre];
      minlim = X.minlim;
      lim_mine = len;
      const int qi = 2 * (lane & (kHalf - 1)) + half;
      if (minlim < len && qi < nq) lim_mine = entry_limit(a.view_limit, X.m.ref_entry[qi / G], len);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_empty[par]);  // this warp has read the hand-off
#pragma unroll
    for (int j = 0; j < kHalf; ++j) l[j] = 0.f;
    ref_mine = (lane & (kHalf - 1)) < nh ? -FLT_MAX : INFINITY;
    bool started = false;  // O holds a tile of this segment
    for (; i < i_end; i += 2) {
      const int buf = (i >> 1) & 1, t = i + t0;
      const uint32_t sw = sw_next;
      sw_next = scales_of(i + 2);
      // A value of zeros (scales are 0 or at least 2^-100) weighs like any other in l, and
      // is taken at 2^-101 in O and the references: below every other, whose precision it would
      // take.  A scale below 2^-8 is "far": another one's up to 2^98 may have put w below fp32's range
      // while the token's share of l counts (2^-24 and up), so l takes it without the scale.
      // With a NaN scale the scores are NaN, and rv is not: a column that masks the token adds 0 rv.
      const float vs = fp4_v_scale(sw);
      const float ks = fp4_k_scale(sw) * q_mul, lv = vs < 0x1p-100f ? -101.f : __log2f(vs);
      const bool far = lv < -8.f;
      const float rv = far ? 0.f : vs >= 0x1p-8f ? __fdividef(1.f, vs) : 1.f;
      // (voted here: a vote beside its use cost 16K tokens 1.042 ms a step where this is 1.014, a
      // ragged batch 12.41 where this is 12.58; an offset in the exponents of all, 1.060 and 12.81)
      const bool any_far = __any_sync(0xffffffffu, far);
      idle_wait(S, a, &S.s_full[st], (i >> 1) & 1);
      tc_fence_after();
      // scores in log2 units with the value's scale in them
      float e[kHalf];
      {
        uint32_t r[kQParts][kHalf];
#pragma unroll
        for (int k = 0; k < kQParts; ++k) tmem_ld16(tl + st * kSCols + k * kN + half * kHalf, r[k]);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kHalf; j += 2) {
          float2 v = as_pair(r[kQParts - 1][j], r[kQParts - 1][j + 1]);
#pragma unroll
          for (int k = kQParts - 2; k >= 0; --k)
            v = __ffma2_rn(v, make_float2(0.0625f, 0.0625f), as_pair(r[k][j], r[k][j + 1]));
          v = __ffma2_rn(v, make_float2(ks, ks), make_float2(lv, lv));
          e[j] = v.x;
          e[j + 1] = v.y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.s_empty[st]);
      if (kLimit && (t + 1) * kT > minlim) {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          const int lim = __shfl_sync(0xffffffffu, lim_mine, j);
          if (t * kT + row >= lim) e[j] = -INFINITY;
        }
      }
      if ((t + 1) * kT > len) {  // the block ends in this tile
#pragma unroll
        for (int j = 0; j < kHalf; ++j) e[j] = t * kT + row < len ? e[j] : -INFINITY;
      }
      auto add_refs = [&](float sign) {
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < kHalf; j += 4) {
          const float4 f = neg_ref[j / 4];
          const float2 v0 = __ffma2_rn(make_float2(f.x, f.y), make_float2(sign, sign), make_float2(e[j], e[j + 1]));
          const float2 v1 = __ffma2_rn(make_float2(f.z, f.w), make_float2(sign, sign), make_float2(e[j + 2], e[j + 3]));
          e[j] = v0.x;
          e[j + 1] = v0.y;
          e[j + 2] = v1.x;
          e[j + 3] = v1.y;
          most = max3(max3(most, v0.x, v0.y), v1.x, v1.y);
        }
        return most;
      };
      // The references move only when some weight would pass 2^(kLift + kLazy), so O
      // is rarely touched; the 128 threads of a half decide together (at a segment's first
      // tile there is nothing to decide).
      bool move = true;
      if (started) move = vote_128(bar, add_refs(1.f) > kLift + kLazy);
      if (move) {
        if (started) add_refs(-1.f);
        float v[kHalf];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) v[j] = e[j];
        max_columns(v, lane);
        float(*red)[4] = S.red[st][half][(i >> 1) & 1];
        if (lane < kHalf) red[lane][qd] = v[0];
        asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
        const float4 t4 = *reinterpret_cast<const float4 *>(red[lane & (kHalf - 1)]);
        const float tmax = fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w));
        const float old = ref_mine;
        if (tmax - old > kLift + kLazy) ref_mine = tmax - kLift;
        const float half_mine = ref_mine == old ? 1.f : ex2(0.5f * (old - ref_mine));
        if (lane < kHalf) S.neg_ref[warp][lane] = -ref_mine;
        if (started) {
#pragma unroll
          for (int j = 0; j < kHalf; ++j) l[j] = l_shrink(l[j], __shfl_sync(0xffffffffu, half_mine, j));
          const float a_mine = half_mine * half_mine;
          // O must hold the stream's earlier tiles before it is rescaled
          idle_wait(S, a, &S.p_empty[st][buf ^ 1], ((i - 2) >> 2) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {  // 8 columns of the first parts, 8 more, then of the second ones
            const uint32_t col = tl + kTmemO + (par * 2 + st) * 2 * kN + (h >> 1) * kN + half * kHalf + (h & 1) * 8;
            uint32_t o[8];
            tmem_ld8(col, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o[j] = __float_as_uint(__uint_as_float(o[j]) * __shfl_sync(0xffffffffu, a_mine, (h & 1) * 8 + j));
            tmem_st8(col, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        add_refs(1.f);
      }
      started = true;
      // weights: their sum, and their parts to the tensor cores
      const __half2 dither = weight_dither(t * kT + row);
      if (any_far) {
        const float back = far ? -lv : -INFINITY;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) l[j] += ex2(e[j] + back);
      }
      uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (4 * c < nh) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = 4 * c + 2 * k;
            const float w0 = ex2(e[j]), w1 = ex2(e[j + 1]);
            const float2 s = __ffma2_rn(make_float2(w0, w1), make_float2(rv, rv), make_float2(l[j], l[j + 1]));
            l[j] = s.x;
            l[j + 1] = s.y;
            uint16_t wh, wl;
            split_weights(w0, w1, dither, wh, wl);
            hi[c] |= static_cast<uint32_t>(wh) << (16 * k);
            lo[c] |= static_cast<uint32_t>(wl) << (16 * k);
          }
        }
      }
      if (i >= 4) idle_wait(S, a, &S.p_empty[st][buf], ((i - 4) >> 2) & 1);  // PV of the buffer's last tile
      st_shared_v4(p_hi + buf * kPBytes, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(p_lo + buf * kPBytes, lo[0], lo[1], lo[2], lo[3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[st][buf]);
      if (pend >= 0) {  // records of the segment before, a tile late
        segment_records(a, S, tmem, pend);
        pend = -1;
      }
    }
    // (before this segment's hand-over: the other stream writes to the same places only
    // once both are done with the segment before)
    if (pend >= 0) segment_records(a, S, tmem, pend);
    sum_columns(l, lane);
    if (lane < kHalf) {
      S.hl[par][st][qd][half * kHalf + lane] = l[0];
      if (qd == 0) S.hm[par][st][half * kHalf + lane] = ref_mine;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.hand[par]);
    pend = seg;
    if (lane == 0) {
      UnitPos x = S.walk[warp];
      S.due[warp] = {seg_id(P, x.b, x.g, x.h), nq, i_end - i0, i0 & 1};
      x.t = x.tiles - 1;
      unit_pos_next(P, a.n_blocks, x);
      S.walk[warp] = x;
    }
    __syncwarp();
    i0 = i_end;
  }
  if (pend >= 0) segment_records(a, S, tmem, pend);
}

// The plan into shared memory (around the RoPE table, which is the launch's own).
__device__ __forceinline__ void issue_plan_copies(const DecodeArgs &a, Fp4Smem &S) {
  constexpr uint32_t kTail = sizeof(PlanShared) - kPhaseOff - kPhaseBytes;
  const uint8_t *src = a.plan + kPlanHeaderBytes;
  uint8_t *dst = reinterpret_cast<uint8_t *>(&S.ps);
  mbar_arrive_expect_tx(&S.plan_bar, sizeof(PlanHeader) + kPhaseOff + kTail + sizeof(CtaPlan));
  bulk_g2s(&S.hdr, a.plan, sizeof(PlanHeader), &S.plan_bar);
  if (kPhaseOff) bulk_g2s(dst, src, kPhaseOff, &S.plan_bar);
  bulk_g2s(dst + kPhaseOff + kPhaseBytes, src + kPhaseOff + kPhaseBytes, kTail, &S.plan_bar);
  bulk_g2s(&S.cp, plan_cta_record(a.plan, blockIdx.x), sizeof(CtaPlan), &S.plan_bar);
}

// Each CTA's share of an array read early by all, into L2.
__device__ __forceinline__ void warm_l2(const void *p, uint64_t total) {
  const uint64_t per = ((total + gridDim.x - 1) / gridDim.x + 255) & ~static_cast<uint64_t>(255);
  const uint64_t off = per * blockIdx.x;
  if (off < total) {
    const uint32_t n = static_cast<uint32_t>(total - off < per ? total - off : per);
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const uint8_t *>(p) + off), "r"(n)
                 : "memory");
  }
}

template <bool kAppend, bool kLimit>
__global__ void __launch_bounds__(kThreads, 1)
    decode_fp4_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  Fp4Smem &S = *reinterpret_cast<Fp4Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // As the other tensor-core kernel (a programmatic dependent of the launch before, see
  // there): before griddepcontrol.wait nothing is written, and nothing read but an L2
  // prefetch and, under the early-loads promise, the plan and the first tiles.
  if (tid == 0) {
    mbar_init(&S.plan_bar, 1);
    fence_mbar_init();
    if (a.early) issue_plan_copies(a, S);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&S.kv_full[s], 1);
      mbar_init(&S.kv_empty[s], 1);
    }
    for (int k = 0; k < 4; ++k) {
      mbar_init(&S.p_full[k >> 1][k & 1], 8);  // the stream's warps
      mbar_init(&S.p_empty[k >> 1][k & 1], 1);
      mbar_init(&S.rec_ready[k], kSoftWarps);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&S.s_full[k], 1);
      mbar_init(&S.s_empty[k], 8);
      mbar_init(&S.mma_done[k], 1);
      mbar_init(&S.q_full[k], 1);
      mbar_init(&S.q_empty[k], 1 + kSoftWarps);  // the segment's last QK, the softmax warps' reads
      mbar_init(&S.o_full[k], 1);
      mbar_init(&S.o_empty[k], kSoftWarps);
      mbar_init(&S.hand[k], kSoftWarps);
    }
    mbar_init(&S.app_bar, 1);
    S.abort_flag = 0;
    S.plan_ok = 1;
    fence_mbar_init();
  }
  if (tid >= 64 && tid < 128) S.ps.cache.phase[tid - 64] = a.phase[tid - 64];
  if (warp == kWarpQk) {
    tmem_alloc(&S.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (tid == 32) warm_l2(a.q, static_cast<uint64_t>(a.n_rows) * a.n_q_heads * 256);
  if (kAppend && tid == 96) {
    warm_l2(a.k_new, static_cast<uint64_t>(a.n_rows) * a.n_kv_heads * 256);
    warm_l2(a.v_new, static_cast<uint64_t>(a.n_rows) * a.n_kv_heads * 256);
  }
  bool plan_timeout = false;
  auto get_plan = [&]() {
    if (tid == 0 && !a.early) issue_plan_copies(a, S);
    __syncthreads();  // the barriers are initialised
    if (!mbar_wait(&S.plan_bar, 0)) {
      plan_timeout = true;
      S.plan_ok = 0;
    }
    if (tid == 0 && !header_matches(a, S.hdr, static_cast<int>(gridDim.x))) S.plan_ok = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  Producer prod;
  prod.count = 0;
  const bool producer = warp == kWarpTma && lane == 0;
  if (a.early) {
    get_plan();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (producer && S.plan_ok && S.cp.u0 < S.cp.u1) {
      // the first tiles into the empty ring (not from the first one with a new token on)
      const int n = static_cast<int>(S.cp.u1 - S.cp.u0);
      start(a, S, prod);
      produce(a, S, &tm_k, &tm_v, prod, n, kAppend && S.cp.app_n > 0 ? S.cp.app_tile : n + kLead, kSlots, -1);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!a.early) {
    get_plan();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (producer && S.plan_ok && S.cp.u0 < S.cp.u1) start(a, S, prod);
  }
  if (plan_timeout) flag_error(a.err, HW_DEV_TIMEOUT);
  const uint32_t tmem = S.tmem_base;
  const bool ok = S.plan_ok != 0;
  if (!ok && tid == 0 && blockIdx.x == 0) flag_error(a.err, HW_DEV_BAD_PLAN);
  const int64_t u0 = ok ? S.cp.u0 : 0, u1 = ok ? S.cp.u1 : 0;
  if (u0 < u1) {
    const int n = static_cast<int>(u1 - u0);
    const bool appending = kAppend && S.cp.app_n > 0;
    if (warp == kWarpTma) {
      if (producer) {
        produce(a, S, &tm_k, &tm_v, prod, n, n + kLead, INT32_MAX, appending ? S.cp.app_tile : -1);
        drain(S, prod);
      }
    } else if (warp == kWarpQk || warp == kWarpPv) {
      if (warp == kWarpQk)
        qk_issuer(a, S, tmem, u0, n);
      else
        pv_issuer(a, S, tmem, u0, n);
      // (no product may be under way when the CTA retires)
      if (elect_one()) mma_commit(&S.mma_done[warp - kWarpQk]);
      __syncwarp();
      mbar_wait(&S.mma_done[warp - kWarpQk], 0);
    } else if (warp == kWarpQ) {
      if (appending) append_tokens(a, S, u0, u1);
      qprep<kLimit>(a, S, u1);
    } else {
      query_prologue(a, S);
      softmax_role<kAppend, kLimit>(a, S, tmem, u0, n);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpQk) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // the merge's 256 threads; its scratch lies in the ring, which nothing uses any more
  if (ok && warp < 8)
    merge_phase<__nv_bfloat16, 128, 8, true>(a, S.ps.plan, S.ps.cache, *reinterpret_cast<MergeSmem<8> *>(S.ring[0]),
                                             &S.cp.mpre[0][0], S.cp.mpre_n, kPreItems, kPreList, tid, 256,
                                             NamedSync<5, 256>(), a.wait_limit, S.cp.mrank,
                                             merge_ctas(a, static_cast<int>(gridDim.x)));
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                              cudaStream_t s) {
  // (kv_scale may be null where there is no token: check_kv_scale)
  if (ctas > 256 || !a.plan || (a.k_new && a.view_limit)) return cudaErrorInvalidValue;
  void (*const kernel)(DecodeArgs, CUtensorMap, CUtensorMap) =
      a.k_new ? decode_fp4_kernel<true, false> : a.view_limit ? decode_fp4_kernel<false, true> : decode_fp4_kernel<false, false>;
  constexpr int kSmem = static_cast<int>(sizeof(Fp4Smem) + 1024);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, tk, tv);
}

}  // namespace hw
