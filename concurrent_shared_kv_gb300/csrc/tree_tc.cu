// tree_tc.cu - attention for trees of drafted tokens on the sm_100 tensor
// cores (tcgen05 + TMEM): bf16 and E4M3 caches with head_dim 128.
//
// A group (hw_tree.h) puts up to 256 query columns (nodes x q heads of a kv
// head x rows that share blocks) against its spans' tokens, as two query tiles
// of 128 rows that share every K/V tile:
//   S [128 queries x 128 tokens] = Q~ . K^T     (A, B in shared memory; Q~ in two parts)
//   O [128 queries x 128 d]     += P . V        (A = P in TMEM)
// With a query per TMEM lane, a softmax thread owns its row: no exchange for
// maxima and sums, and P goes back to the columns that S came from.
//
// The CTA runs two streams, each with its own S/P, O, issuing warp and eight
// softmax warps: with over 128 columns stream q is query tile q and both take
// every K/V tile; with up to 128 there is one query tile and the streams take
// the K/V tiles by turns (two records, like two CTAs).  One stream's products
// run under the other's softmax; within a stream QK, softmax and PV follow one
// another (S and P share their columns: TMEM holds no third score tile), so
// what counts is the length of that chain.  Two threads share a row, 64 tokens
// each, and exchange their maxima.
// What bounds it: a tile of 128 tokens against 256 columns needs 3100 clocks of
// the tensor cores (QK over both parts of Q~; E4M3 2100) and takes about 3800:
// the chain, and a ring of three stages beside two query tiles of two parts.
// Against 128 columns it is 1536 and about 1700, of which the DRAM needs 2400
// where every tile is new.  A new span costs 6000 or more: its queries are
// loaded, turned and written while the tensor cores wait.  Measured, a layer
// with its writes and merge: 4 trees of 64 nodes over 16K tokens (40/8 heads)
// 117 us, the tensor cores busy for 68 %; of 16 nodes 43 us; 8 x 4 ragged trees
// of 8 nodes over up to 32K tokens 141 to 157 us, 4.6 to 5.2 TB/s; E4M3, 4 trees
// of 24 nodes over 32K tokens (32/8 heads) 65 us.  (With Q~ in one part, half
// the QK products and five stages: 93, 39.6 and 139 to 163 us.)
// Warps: 0-7 softmax of stream 0 (0-3 tokens 0-63, 4-7 the others), 8-15 of
// stream 1, 16 the TMA producer, 17 and 18 the issuers.
// Rotated queries carry scale * log2(e), so scores leave the MMA in log2
// units.  They are held as two bf16 parts, hi and what that leaves, as the
// decode holds them: a score keeps 16 bits, and QK runs over both.  P is rounded
// to bf16 once, as the decode's is, against sums of weights in fp32.  Outputs
// are measured 0.0015 to 0.0016 off the exact result in the 2-norm, which is the
// output's own rounding; 0.0024 where 60000 tokens of unlike values share the
// weight, P's rounding beside it.  (With queries rounded to bf16 once it was
// 0.0033, and more for larger scores: the error of a score grows with it, that of
// a weight does not.)
//
// E4M3 caches: both products run as kind::f8f6f4 on the codes, at twice the
// rate, with Q~ and P each as two E4M3 parts x = hi + lo, lo the rounded
// remainder (half a step 2^-4 twice: 2^-8, bf16's), summed into the same
// accumulator.  A query is scaled by a power of two that brings its largest
// element into [128, 256), and takes its kv head's k_scale along; its scores
// are scaled back in the softmax.  P is kept 2^4 times larger than the running
// maximum asks for (below 2^8 until O is rescaled, E4M3 ends at 448), so that
// weights down to 2^-10 keep both parts' full precision; the factor is in the
// record's m.  (2^6: error 0.00219 instead of 0.00223, but O was rescaled
// wherever a maximum grew by 2^2, and 4 trees of 24 nodes over 32K tokens took
// 79 us where they now took 71.5.)
#include <cuda.h>
#include <cuda_fp16.h>

#include "hw_device.cuh"
#include "hw_sm100.cuh"
#include "hw_tree.h"

namespace hw {

using namespace sm100;

namespace {

constexpr int kThreads = 608;
constexpr int kWarpTma = 16, kWarpMma = 17;  // and 18: an issuer a stream
constexpr int kT = 128;                      // tokens per tile
constexpr uint32_t kBox = 128 * 128;         // 128 rows of 128 bytes, 128-byte swizzled
// The ring of K and V tiles: bf16 two boxes each, E4M3 one.  A CTA without a
// group of over 128 columns has no second query tile, and that much more ring
// (kMore stages): what one query tile can do is bound by the bytes under way.
template <bool kFp8>
struct Ring {
  static constexpr uint32_t kQTile = kFp8 ? 2 * kBox : 4 * kBox;  // a query tile: hi, then lo; bf16 d 0-63 and d 64-127 of each
  static constexpr uint32_t kStage = kFp8 ? kBox : 2 * kBox;
  static constexpr int kStages = kFp8 ? 9 : 3;
  static constexpr int kMore = kQTile / kStage;
  static constexpr int kStep = kFp8 ? 32 : 16;  // tokens of one MMA
  // A wait for a stage's next tile can be told from its last one only if that
  // has landed.  A stream that has waited for turn m - 1 of the other one knows
  // that the V tiles of that one's turns up to m - 3 have landed, and those of
  // its own up to m - 4.  Three stages before the K of tile t is the V of tile
  // t - 2, its turns at least three and four before tile t's where both streams
  // take every tile, as they do wherever the ring has fewer stages than five;
  // five before it, in the order of KvPos, that of tile t - 4, four turns back.
  static_assert(kStages >= 3 && kStages + kMore >= 5, "the barriers' phases");
};
// A place in a ring of n stages.
struct RingPos {
  int s;
  uint32_t phase;
  __device__ __forceinline__ void on(int by, int n) {
    s += by;
    if (s >= n) {
      s -= n;
      phase ^= 1;
    }
  }
};
// Where the CTA's tiles are in the ring.  Where streams take turns the V of
// tile t is used with the K of tile t + 2, and where that makes a difference
// (`ahead`) the ring is filled in that order, K(0) K(1) V(0) K(2) V(1) .. V(n-1):
// a place then is not held up by one that is used later.  Else K(0) V(0) K(1) ..
struct KvPos {
  RingPos k, v;
  int left, stages;  // tiles from this one on
  bool ahead, first;
  __device__ __forceinline__ KvPos(int n, int ring, bool a) : k{0, 0}, v{0, 0}, left(n), stages(ring), ahead(a), first(true) {
    v.on(ahead && n > 1 ? 2 : 1, stages);
  }
  __device__ __forceinline__ void next() {
    k.on(ahead && first ? 1 : 2, stages);
    v.on(ahead && left == 2 ? 1 : 2, stages);
    first = false;
    --left;
  }
};
constexpr float kLazy = 8.f;                 // O is rescaled only when a weight would pass 2^8
constexpr float kLift = 4.f;                 // E4M3: log2 of P's factor
constexpr uint32_t kTmemCols = 512;          // S0/P0, S1/P1, O0, O1: 128 columns each

template <bool kFp8>
struct TcSmem {
  static constexpr int kStages = Ring<kFp8>::kStages;
  static constexpr int kAll = kStages + Ring<kFp8>::kMore;
  alignas(1024) uint8_t q[2][Ring<kFp8>::kQTile];                     // (the second tile's place: part of the ring without one)
  alignas(1024) uint8_t kv[kStages][Ring<kFp8>::kStage];
  uint64_t kv_full[kAll], kv_empty[kAll];
  uint64_t q_full[2], q_free, s_full[2], p_half[2], p_full[2], pv_done[2], o_empty[2], order, mma_done;
  // tidied V tiles, by the stream that does it, alternating; the tokens with a value that is not finite
  uint64_t scanned[2][2];
  uint32_t bad[2][2][2][4];
  float red[2][2][128];  // per stream: the maxima of a row's halves (at a record: sums)
  float back[kFp8 ? 2 : 1][2][kFp8 ? 128 : 1];  // E4M3: per span parity and query tile, the rows' score factors
  uint32_t tmem;
  int32_t abort_flag;
};
static_assert(sizeof(TcSmem<false>) <= 232448 && sizeof(TcSmem<true>) <= 232448, "shared memory of one CTA per SM");

template <typename Smem>
__device__ __forceinline__ bool aborted(Smem &S) {
  return *reinterpret_cast<volatile int32_t *>(&S.abort_flag) != 0;
}
// Wait with a bound; false once the CTA winds down.
template <typename Smem>
__device__ __forceinline__ bool wait_or_abort(Smem &S, const TreeArgs &a, uint64_t *bar, uint32_t parity) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_test(bar, parity)) {
    if (aborted(S)) return false;
    if (clock64() - t0 > kWaitLimit) {
      *reinterpret_cast<volatile int32_t *>(&S.abort_flag) = 1;
      flag_error(reinterpret_cast<int32_t *>(a.ws), HW_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

// wait_or_abort by a whole warp, with one answer for all its lanes: what
// follows are warp-wide TMEM accesses.
template <typename Smem>
__device__ __forceinline__ bool warp_wait(Smem &S, const TreeArgs &a, uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_or_abort(S, a, bar, parity));
}
// The same for the softmax warps: suspended while they wait.  (Sixteen warps
// that poll take the issue slots of those that compute.)
template <typename Smem>
__device__ __forceinline__ void idle_wait(Smem &S, const TreeArgs &a, uint64_t *bar, uint32_t parity) {
  if (!mbar_try(bar, parity)) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
      if (aborted(S)) break;
      if (clock64() - t0 > kWaitLimit) {
        *reinterpret_cast<volatile int32_t *>(&S.abort_flag) = 1;
        flag_error(reinterpret_cast<int32_t *>(a.ws), HW_DEV_TIMEOUT);
        break;
      }
    }
  }
  __syncwarp();
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs, fp32 accumulator.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// 32 lanes x 8 columns.
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

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}
// (x, y) in bf16, and what that leaves of them, in bf16 too.  (An infinity
// leaves NaN, as its products with values of both signs do.)
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(x, y);
  lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
// The same for 8-bit inputs.
__device__ __forceinline__ void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two fp16 numbers as E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
// (x, y), at most 256, as two E4M3 parts each: hi and lo = x - hi, two codes in
// each.  fp16 in between keeps 11 bits, more than the parts do together; hi is
// cut to E4M3's 3 bits behind the leading one there (ties away), so no code
// has to be turned back.  (Below 2^-6, where E4M3 has fewer bits, hi's code is
// rounded once more: 2^-10 at most, beside a largest value of 2^6 and up.)
__device__ __forceinline__ void split_e4m3(float x, float y, uint32_t &hi, uint32_t &lo) {
  const __half2 v = __floats2half2_rn(x, y);
  const uint32_t top = (*reinterpret_cast<const uint32_t *>(&v) + 0x00400040u) & 0xff80ff80u;
  hi = e4m3x2(top);
  const __half2 rest = __hsub2(v, *reinterpret_cast<const __half2 *>(&top));
  lo = e4m3x2(*reinterpret_cast<const uint32_t *>(&rest));
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&x)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// The CTA's units, span by span.
struct Walk {
  const TreeArgs &a;
  int streams;
  int head, group, span, tile, left;  // kv head, group, span, its first tile, units still to come
  TreeGroup g;
  TreeSpan sp;
  int tiles;  // of this span that are the CTA's
  int stages;     // of the ring
  bool ahead;     // how it is filled (KvPos)
  uint32_t ring;  // its shared-memory address
  __device__ __forceinline__ void load_span() {
    sp = tree_at<TreeSpan>(a, a.L.spans)[g.span0 + span];
    begin();
  }
  __device__ __forceinline__ void begin() {
    prefetch_l1(tree_at<TreeSpan>(a, a.L.spans) + g.span0 + span + 1);
    tiles = min((sp.len + kT - 1) / kT - tile, left);
  }
  // On to the next span: 0 at the end, 1 in the same group, 2 in another one.
  __device__ __forceinline__ int next() {
    left -= tiles;
    if (left <= 0) return 0;
    tile = 0;
    const bool other = ++span == g.n_spans;
    if (other) {
      span = 0;
      next_group(*tree_at<const TreeHeader>(a, a.L.hdr), head, group);
      g = tree_at<TreeGroup>(a, a.L.groups)[group];
    }
    load_span();
    return other ? 2 : 1;
  }
};

template <bool kFp8>
__device__ void producer(const TreeArgs &a, TcSmem<kFp8> &S, const CUtensorMap *tk, const CUtensorMap *tv, Walk w) {
  constexpr uint32_t kStage = Ring<kFp8>::kStage;
  const uint64_t pol = policy_evict_first();
  uint8_t *ring = w.stages > Ring<kFp8>::kStages ? S.q[1] : S.kv[0];
  int n = 0;  // ring entries issued: K(0), V(0), K(1), V(1), ...
  RingPos at = {0, 0};
  bool waited = false, go = true;
  auto load = [&](bool v, int row, int head) {
    if (n >= w.stages && !wait_or_abort(S, a, &S.kv_empty[at.s], at.phase ^ 1)) return false;
    uint8_t *to = ring + at.s * kStage;
    mbar_arrive_expect_tx(&S.kv_full[at.s], kStage);
    tma_load_3d(to, v ? tv : tk, &S.kv_full[at.s], 0, row, head, pol);
    if constexpr (!kFp8) tma_load_3d(to + kBox, v ? tv : tk, &S.kv_full[at.s], 64, row, head, pol);
    ++n;
    at.on(1, w.stages);
    return true;
  };
  int v_row = -1, v_head = 0;  // the V behind the next K, if any
  do {
    if (w.sp.row >= 0 && !waited) {  // a tree: its tokens come from the launch before
      asm volatile("griddepcontrol.wait;" ::: "memory");
      asm volatile("fence.proxy.async;" ::: "memory");
      waited = true;
    }
    // what the softmax warps look up first when they get to this span (a trip
    // to L2 there holds up everything)
    if (w.sp.row < 0) {
      prefetch_l1(tree_at<int16_t>(a, a.L.map) + w.sp.map);
    } else {
      const uint2 *mask = tree_at<uint2>(a, a.L.mask) + 2 * static_cast<int64_t>(w.sp.row) * a.max_nodes;
      for (int i = 0; i < w.sp.len; i += 8) prefetch_l1(mask + 2 * i);
    }
    for (int t = w.tile; go && t < w.tile + w.tiles; ++t) {
      const int row = w.sp.start + t * kT;
      go = load(false, row, w.head);
      if (w.ahead) {
        if (go && v_row >= 0) go = load(true, v_row, v_head);
        v_row = row;
        v_head = w.head;
      } else if (go) {
        go = load(true, row, w.head);
      }
    }
  } while (go && w.next());
  if (go && v_row >= 0) load(true, v_row, v_head);
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
  // no copy may still be landing when the CTA retires
  RingPos back = {0, 0};
  if (n >= w.stages) back = {at.s, at.phase ^ 1};
  for (int j = min(n, w.stages); j > 0; --j, back.on(1, w.stages)) mbar_wait(&S.kv_full[back.s], back.phase);
}

// One stream's products.  The whole warp walks and waits; one elected lane
// issues.  (Descriptors then stay in uniform registers: issued from a branch
// of one lane, 8 MMAs took 1200 clocks instead of the 512 the tensor cores
// need for them.  Even so a tile's waits and 16 MMAs keep a warp busy for
// 1700 clocks, which is why each stream has its own.)
template <bool kFp8>
__device__ void mma_issuer(const TreeArgs &a, TcSmem<kFp8> &S, uint32_t tmem, Walk w, int q) {
  constexpr int kStep = Ring<kFp8>::kStep;
  constexpr int kSteps = kFp8 ? 8 : 16;  // of QK: 128 d, 32 or 16 a step, hi and lo
  constexpr uint32_t kStage = Ring<kFp8>::kStage;
  constexpr uint32_t idesc_qk = kFp8 ? idesc_e4m3(128, 128, 0, 0) : idesc_bf16(128, 128, 0, 0);
  constexpr uint32_t idesc_pv = kFp8 ? idesc_e4m3(128, 128, 0, 1) : idesc_bf16(128, 128, 0, 1);
  const uint32_t q0 = smem_u32(S.q[0]), kv0 = w.ring;
  const uint64_t a_qk = smem_desc(q0, 16, 1024, kSw128), b_qk = smem_desc(kv0, 16, 1024, kSw128);
  const uint64_t b_pv = smem_desc(kv0, kBox, 1024, kSw128);
  const uint32_t s_tmem = tmem + q * 128, o_tmem = s_tmem + 256;
  int np = 0, no = 0, nspan = 0;  // PVs issued, groups whose PVs have begun, spans
  // the tile whose PV is to come, if any: its V's place, its steps of kStep
  // tokens, whether it is the stream's first of a group
  RingPos pend_v = {0, 0};
  int pend_steps = 0;
  bool pend = false, pend_first = false, pend_two = false, first = true;
  // Everything but P is waited for first: P is what the products wait for.  It
  // comes in two parts, the first 32 tokens of each half of the tile before
  // the others; the first part's products run while the second is computed.
  auto pv_ready = [&]() -> bool {
    return warp_wait(S, a, &S.kv_full[pend_v.s], pend_v.phase) &&
           (!pend_first || warp_wait(S, a, &S.o_empty[q], (no++ & 1) ^ 1)) &&
           warp_wait(S, a, &S.p_half[q], np & 1);
  };
  auto pv_part = [&](int part) {  // by the elected lane
    const uint64_t bs = b_pv + ((pend_v.s * kStage) >> 4);
#pragma unroll
    for (int k = 0; k < 128 / kStep; ++k)
      if (((k * kStep >> 5) & 1) == part && k < pend_steps) {
        const uint64_t b = bs + ((k * kStep * 128) >> 4);
        // (each half of the tokens has its weights in the first columns of its scores')
        const uint32_t p = s_tmem + (k * kStep >= 64 ? 64 + (k * kStep - 64) / (kFp8 ? 4 : 2) : k * kStep / (kFp8 ? 4 : 2));
        if constexpr (kFp8) {
          mma_f8_ts(o_tmem, p, b, idesc_pv, !(pend_first && k == 0));
          mma_f8_ts(o_tmem, p + 16, b, idesc_pv, true);
        } else {
          mma_bf16_ts(o_tmem, p, b, idesc_pv, !(pend_first && k == 0));
        }
      }
  };
  auto pv_first = [&]() -> bool {
    if (!pv_ready()) return false;
    tc_fence_after();
    if (elect_one()) pv_part(0);
    __syncwarp();
    return warp_wait(S, a, &S.p_full[q], np & 1);
  };
  auto pv = [&]() {  // what is left of them, by the elected lane
    const int s = pend_v.s;
    pv_part(1);
    mma_commit(&S.pv_done[q]);
    mma_commit(&S.kv_empty[s]);
    if (!pend_two) mma_commit(&S.kv_empty[s]);  // (for the other stream, which does not use it)
  };
  // The products that end a group, outside the order of the others.
  auto flush = [&]() -> bool {
    if (!pv_first()) return false;
    tc_fence_after();
    if (elect_one()) pv();
    __syncwarp();
    ++np;
    pend = false;
    return true;
  };
  // The span's queries; one query tile is written by all softmax warps.
  // (This stream's first: once they are there the other issuer has seen the
  // other stream's of the span before.)
  auto queries = [&](bool two) -> bool {
    return warp_wait(S, a, &S.q_full[q], nspan & 1) && (two || warp_wait(S, a, &S.q_full[q ^ 1], nspan & 1));
  };
  KvPos at(w.left, w.stages, w.ahead);
  int step = 2;         // 2: a group starts
  // Turns at the tensor cores so far, of both streams.  They alternate over the
  // whole of the CTA's work, stream 0 the even ones: whoever waits for the turn
  // before its own has made the one before that, so a bit tells them apart.
  int turns = 0;
  bool go = true;
  do {
    const bool two = w.g.n_cols > 128;
    if (step == 2) {  // the softmax warps wait for a group's last products
      if (pend && !(go = flush())) break;
      first = true;
    }
    bool turned = false;  // this span's queries are there
    for (int t = 0; t < w.tiles; ++t, at.next(), turns += two ? 2 : 1) {
      const bool later = (turns ^ q) & 1;  // the other stream's turn is before this one's
      if (!two && later) continue;
      const int s = at.k.s, mine = turns + later;
      // (a new span's queries come after the last P, so their wait is last)
      // One stream's PV and QK go out together, the streams in turn: mixed,
      // both would wait for both, and their softmaxes would run at the same
      // time, the tensor cores idle.
      if (mine > 0 && !(go = warp_wait(S, a, &S.order, (mine - 1) & 1))) break;
      // Not before the turn: it says that the stage's last tile has landed (Ring).
      // (With three stages the next K comes into the place of the V before the
      // pending one: the pending products do not wait for it.)
      if (w.stages < 5 && pend && !(go = flush())) break;
      if (!(go = warp_wait(S, a, &S.kv_full[s], at.k.phase))) break;
      if (pend && !(go = pv_first())) break;
      if (!turned && !(go = queries(two))) break;
      turned = true;
      tc_fence_after();
      const uint64_t as = a_qk + ((two ? q * Ring<kFp8>::kQTile : 0) >> 4), bs = b_qk + ((s * kStage) >> 4);
      if (elect_one()) {
        if (pend) pv();
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {  // over d with hi, then with lo
          const uint32_t o = ((j >> 2) * kBox + (j & 3) * 32) >> 4;
          if constexpr (kFp8)
            mma_f8(s_tmem, as + o, bs + (((j & 3) * 32) >> 4), idesc_qk, j > 0);
          else
            mma_bf16(s_tmem, as + o, bs + ((((j >> 2) & 1) * kBox + (j & 3) * 32) >> 4), idesc_qk, j > 0);
          if (j == kSteps - 3) mbar_arrive(&S.order);  // (the next turn's first MMA is two MMAs away)
        }
        mma_commit(&S.s_full[q]);
        mma_commit(&S.kv_empty[s]);
        if (!two) mma_commit(&S.kv_empty[s]);
      }
      __syncwarp();
      if (pend) ++np;
      pend = true;
      pend_v = at.v;
      pend_steps = (min(kT, w.sp.len - (w.tile + t) * kT) + kStep - 1) / kStep;
      pend_first = first;
      pend_two = two;
      first = false;
    }
    // (also without a tile: the issuer must not run ahead of the queries)
    if (!go || (!turned && !(go = queries(two)))) break;
    if (elect_one()) mma_commit(&S.q_free);
    __syncwarp();
    ++nspan;
  } while ((step = w.next()));
  if (go && pend) flush();
  if (elect_one()) mma_commit(&S.mma_done);
  __syncwarp();
  mbar_wait(&S.mma_done, 0);
}

// N queries of a warp's 32 (a row each, from `first`), rotated, scaled and
// rounded into the query tile at `to`.  Eight lanes take a query, each 8
// elements and their partners 64 further: every load of a query or of a
// rotation is then one line of memory.  (A thread a query touched 32 lines a
// load and took 8000 clocks for 256 queries.)  src, rot: the query and the
// rotation's table row of this lane's own query, rot < 0: it does not see the
// span, and its row of the tile may hold anything.  back (E4M3): the rows'
// factors that undo their scaling.
template <bool kFp8, int N>
__device__ __forceinline__ void write_queries(const __nv_bfloat16 *q, const uint4 *table, int src, int rot, uint32_t to,
                                              float scale, int first, int lane, float *back) {
  const int c = lane & 7;
  // (rows that see nothing read row 0: loads without branches are all under
  // way before the first is needed, and one trip to L2 costs a thousand
  // clocks or more)
  constexpr int kTurn = kFp8 ? 2 : 4;  // 16-byte pieces of (cos, sin) for 8 elements: fp16, fp32
  uint4 u[N / 4], v[N / 4], cs[N / 4][kTurn];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const int at = first + 4 * i + (lane >> 3);
    const int row = __shfl_sync(0xffffffffu, src, at), turn = max(0, __shfl_sync(0xffffffffu, rot, at));
    const uint4 *x = reinterpret_cast<const uint4 *>(q + static_cast<int64_t>(row) * 128);
    const uint4 *t = table + static_cast<int64_t>(turn) * 8 * kTurn;
    u[i] = __ldg(x + c);
    v[i] = __ldg(x + c + 8);
#pragma unroll
    for (int j = 0; j < kTurn; ++j) cs[i][j] = __ldg(t + c + 8 * j);  // (turn_at)
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, y[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t w[4 * kTurn];
#pragma unroll
    for (int j = 0; j < kTurn; ++j) w[4 * j] = cs[i][j].x, w[4 * j + 1] = cs[i][j].y, w[4 * j + 2] = cs[i][j].z, w[4 * j + 3] = cs[i][j].w;
    float p[8], r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 t = kFp8 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[j]))
                            : make_float2(__uint_as_float(w[(2 * j) % (4 * kTurn)]), __uint_as_float(w[(2 * j + 1) % (4 * kTurn)]));
      const float x0 = __uint_as_float(j & 1 ? x[j / 2] & 0xffff0000u : x[j / 2] << 16);
      const float y0 = __uint_as_float(j & 1 ? y[j / 2] & 0xffff0000u : y[j / 2] << 16);
      p[j] = (x0 * t.x - y0 * t.y) * scale;
      r[j] = (y0 * t.x + x0 * t.y) * scale;
    }
    const int at = first + 4 * i + (lane >> 3);
    const uint32_t o = to + at * 128;
    if constexpr (kFp8) {
      // a power of two brings the largest element into [128, 256)
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max3(top, fabsf(p[j]), fabsf(r[j]));
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      // (exponent of top, at most 2^127; the two factors' product is 1)
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 20), 240);
      const float up = __uint_as_float(static_cast<uint32_t>(254 + 7 - e) << 23);  // 2^(7 - exponent)
      if (c == 0) back[at] = top < INFINITY ? __uint_as_float(static_cast<uint32_t>(e - 7) << 23) : NAN;
      uint32_t hp[4], lp[4], hr[4], lr[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        split_e4m3(p[2 * j] * up, p[2 * j + 1] * up, hp[j], lp[j]);
        split_e4m3(r[2 * j] * up, r[2 * j + 1] * up, hr[j], lr[j]);
      }
      const uint32_t o0 = o + (((c >> 1) ^ (at & 7)) << 4) + (c & 1) * 8, o1 = o + (((4 + (c >> 1)) ^ (at & 7)) << 4) + (c & 1) * 8;
      st_shared_v2(o0, hp[0] | hp[1] << 16, hp[2] | hp[3] << 16);
      st_shared_v2(o1, hr[0] | hr[1] << 16, hr[2] | hr[3] << 16);
      st_shared_v2(o0 + kBox, lp[0] | lp[1] << 16, lp[2] | lp[3] << 16);
      st_shared_v2(o1 + kBox, lr[0] | lr[1] << 16, lr[2] | lr[3] << 16);
    } else {
      const uint32_t oc = o + ((c ^ (at & 7)) << 4);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split_bf16(p[2 * j], p[2 * j + 1], hi[j], lo[j]);
      st_shared_v4(oc, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(oc + 2 * kBox, lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) split_bf16(r[2 * j], r[2 * j + 1], hi[j], lo[j]);
      st_shared_v4(oc + kBox, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(oc + 3 * kBox, lo[0], lo[1], lo[2], lo[3]);
    }
  }
}

// The two warps that share rows (barriers 1 .. 8).
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

// Half of one row's record: 64 of O's columns, 32 bytes of every 8 d side by
// side for the group's columns, so that a warp's stores fill whole sectors.
__device__ __forceinline__ void store_record(const TreeArgs &a, uint32_t o_tmem, int64_t rec, int n_cols, int col,
                                             int half, float scale) {
  float *dst = tree_at<float>(a, a.L.o) + rec * 128 + col * 8 + static_cast<int64_t>(half) * 8 * n_cols * 8;
  const bool on = col < n_cols;
#pragma unroll 4
  for (int c = 0; c < 8; ++c) {
    uint32_t r[8];
    tmem_ld8(o_tmem + 64 * half + 8 * c, r);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 8; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * scale);
    if (on)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + static_cast<int64_t>(c) * n_cols * 8),
                   "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                   : "memory");
  }
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The softmax of a stream.  Its waits give up together (abort_flag), and the
// code then runs on to its end without waiting, on whatever the tiles hold:
// the named barriers in it stay matched.
template <bool kFp8>
__device__ void softmax(const TreeArgs &a, TcSmem<kFp8> &S, uint32_t tmem, Walk w, int q) {
  constexpr int kStep = Ring<kFp8>::kStep;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, half = (threadIdx.x >> 7) & 1;
  const int row = quarter * 32 + lane, pair = 1 + q * 4 + quarter;
  const uint32_t s_tmem = tmem + q * 128 + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t o_tmem = s_tmem + 256;
  int ns = 0;              // tiles of this stream so far
  KvPos at(w.left, w.stages, w.ahead);
  int nspan = 0;           // spans of the CTA so far
  int np0 = 0, np1 = 0;    // tiles tidied by each stream so far
  float m = 0.f, l = 0.f;  // the row's maximum; this half's sum
  // the record to come: that of the group before (0 columns: none)
  int64_t rec = 0;
  int rec_cols = 0, rec_col = 0;
  float rec_scale = 1.f;   // E4M3: its kv head's v_scale
  bool some = false;       // the stream had a tile of it
  auto record = [&]() {
    const bool on = rec_col - lane < rec_cols;  // (the same for the pair's warps)
    if (some) idle_wait(S, a, &S.pv_done[q], (ns - 1) & 1);
    if (on) {
      S.red[q][half][row] = l;
      pair_sync(pair);
      if (half == 0 && rec_col < rec_cols && (some || w.streams == 2))  // a stream without a tile leaves m = -inf and no O
        tree_at<float2>(a, a.L.ml)[rec + rec_col] =
            some ? make_float2(m, l + S.red[q][1][row]) : make_float2(-INFINITY, 0.f);
      pair_sync(pair);
      tc_fence_after();
      if (some) store_record(a, o_tmem, rec, rec_cols, rec_col, half, rec_scale);
    }
    tc_fence_before();
    __syncwarp();
    if (some && lane == 0) mbar_arrive(&S.o_empty[q]);
  };
  int step = 2;
  int turn = 0;  // the stream of the next tile that is one stream's (the issuers' turns)
  do {
    const bool two = w.g.n_cols > 128;
    const int col = two ? q * 128 + row : row;               // the thread's column of the group
    const bool mine = col < w.g.n_cols;                      // a query in this row
    const bool warp_on = col - lane < w.g.n_cols;
    // (loaded again for every span of a group: registers are what is short)
    const int G = a.n_q_heads / a.n_kv_heads;
    const int heads = tree_at<int32_t>(a, a.L.heads)[w.head * G + min(lane, G - 1)];  // the kv head's q heads, a lane each
    TreeColumn tc = {};
    if (mine) tc = tree_at<TreeColumn>(a, a.L.columns)[w.g.col0 + col];
    const int src = tc.node * a.n_q_heads + __shfl_sync(0xffffffffu, heads, tc.head);  // the row's query (row 0 where there is none)
    // the tokens the column sees: all, a node's ancestors and itself, or none
    uint2 see = make_uint2(0, 0);
    int v = -1;
    // (a lane loads a row's entry beside the columns' load, not behind it)
    int entry = -1;
    const bool few = w.g.n_rows <= 32;
    if (w.sp.row < 0 && few && lane < w.g.n_rows) entry = tree_at<int16_t>(a, a.L.map)[w.sp.map + lane];
    entry = __shfl_sync(0xffffffffu, entry, tc.row & 31);
    if (mine) {
      v = w.sp.row < 0 ? few ? entry : tree_at<int16_t>(a, a.L.map)[w.sp.map + tc.row]
          : static_cast<uint32_t>(tc.node - w.sp.row * a.max_nodes) < static_cast<uint32_t>(a.max_nodes) ? a.n_view : -1;
      if (v >= 0) see = w.sp.row < 0 ? make_uint2(~0u, ~0u) : tree_at<uint2>(a, a.L.mask)[2 * static_cast<int64_t>(tc.node) + half];
    }
    // Q~ of the span before is free once its last scores are there
    if (nspan > 0) idle_wait(S, a, &S.q_free, (nspan - 1) & 1);
    if (warp_on) {
      const __nv_bfloat16 *qs = static_cast<const __nv_bfloat16 *>(a.q);
      const uint4 *table = tree_at<uint4>(a, a.L.turns);
      const int rot = v < 0 ? -1 : tc.rot + v * tc.n_nodes;
      // two query tiles: a tile a stream, half of a warp's rows a half; one: a quarter each
      const uint32_t to = smem_u32(S.q[two ? q : 0]) + quarter * 32 * 128;
      const float scale = kFp8 ? a.scale_log2 * a.k_scale[w.head] : a.scale_log2;
      float *back = &S.back[kFp8 ? nspan & 1 : 0][two ? q : 0][kFp8 ? quarter * 32 : 0];
      if (two) {
        constexpr int N = kFp8 ? 16 : 8;  // (as many as registers hold)
#pragma unroll 1
        for (int i = 0; i < 16; i += N) write_queries<kFp8, N>(qs, table, src, rot, to, scale, 16 * half + i, lane, back);
      } else
        write_queries<kFp8, 8>(qs, table, src, rot, to, scale, 8 * (2 * q + half), lane, back);
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_full[q]);
    if (step == 2) {
      if (rec_cols > 0) record();
      const int64_t p = static_cast<int64_t>(w.head) * tree_at<TreeHeader>(a, a.L.hdr)->n_groups + w.group;
      rec_cols = w.g.n_cols;
      rec_col = col;
      if (kFp8) rec_scale = a.v_scale[w.head];
      // one record a CTA, or one a stream
      const int nth = static_cast<int>(blockIdx.x) - tree_at<int2>(a, a.L.piece_cta)[p].x;
      rec = tree_at<int32_t>(a, a.L.piece_row)[p] + static_cast<int64_t>(two ? nth : w.streams * nth + q) * rec_cols;
      some = false;
    }
    ++nspan;
    for (int t = 0; t < w.tiles; ++t, at.next(), turn ^= !two) {
      const int valid = min(kT, w.sp.len - (w.tile + t) * kT);
      const int owner = two ? 0 : turn;  // who tidies the V tile, where that is needed
      const bool tidy = w.sp.partial || (valid & (kStep - 1));
      if (!two && turn != q) {
        if (tidy) ++(owner ? np1 : np0);
        continue;
      }
      idle_wait(S, a, &S.s_full[q], ns & 1);
      bool bad = false;
      if (tidy) {
        const int np = owner ? np1 : np0, par = np & 1;
        const RingPos v = at.v;
        if (q == owner) {
          // 0 * NaN would poison a sum.  V rows past the span, up to the end
          // of the last step of tokens, may hold anything: cleared.  In a
          // tile that not every column sees, so are values that are not
          // finite: the columns that see their token get a NaN through l.
          idle_wait(S, a, &S.kv_full[v.s], v.phase);
          constexpr int kPieces = kFp8 ? 4 : 8;  // 16-byte pieces of a row's half
          const uint32_t at = w.ring + v.s * Ring<kFp8>::kStage + half * (kFp8 ? 64 : kBox) + row * 128;
          const bool clear = row >= valid && row < ((valid + kStep - 1) & ~(kStep - 1));
          bool odd = false;
          if (w.sp.partial && row < valid)
            for (int c = 0; c < kPieces; ++c) {
              uint32_t x[4];
              ld_shared_v4(at + ((c + row) & (kPieces - 1)) * 16, x);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                odd |= kFp8 ? __vcmpeq4(x[j] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0
                            : (x[j] & 0x7f80u) == 0x7f80u || (x[j] & 0x7f800000u) == 0x7f800000u;
            }
          if (clear || odd) {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) st_shared_v4(at + c * 16, 0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          const uint32_t bits = __ballot_sync(0xffffffffu, odd);
          if (lane == 0) {
            S.bad[owner][par][half][quarter] = bits;
            mbar_arrive(&S.scanned[owner][par]);
          }
        }
        idle_wait(S, a, &S.scanned[owner][par], (np >> 1) & 1);
        const uint32_t(*b)[4] = S.bad[owner][par];
        bad = ((b[0][2 * half] | b[1][2 * half]) & see.x) || ((b[0][2 * half + 1] | b[1][2 * half + 1]) & see.y);
        ++(owner ? np1 : np0);
      }
      if (warp_on) {
        tc_fence_after();
        // Half of the row's scores are in registers at a time, those of tokens
        // 32-63 twice: what does not fit there is kept in local memory, for
        // which the shared memory in use leaves next to no L1.
        uint32_t s[32];
        auto load = [&](int c) {
          tmem_ld32(s_tmem + 64 * half + 32 * c, s);
          tmem_wait_ld();
          if (valid < kT || w.sp.partial) {
            const int in = min(32, max(0, valid - 64 * half - 32 * c));
            const uint32_t bits = (c ? see.y : see.x) & (in == 32 ? ~0u : (1u << in) - 1u);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((bits >> j) & 1u)) s[j] = 0xff800000u;  // -inf
          }
        };
        float top = -INFINITY;
#pragma unroll
        for (int c = 1; c >= 0; --c) {
          load(c);
          float mx[2] = {-INFINITY, top};
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            mx[0] = max3(mx[0], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
            mx[1] = max3(mx[1], __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
          }
          top = fmaxf(mx[0], mx[1]);
        }
        // (the partner has read this before the next tile's scores can come)
        S.red[q][half][row] = top;
        pair_sync(pair);
        top = fmaxf(top, S.red[q][half ^ 1][row]);
        const float f = kFp8 ? S.back[kFp8 ? (nspan - 1) & 1 : 0][two ? q : 0][kFp8 ? row : 0] : 1.f;
        if constexpr (kFp8) top *= f;
        constexpr float lift = kFp8 ? kLift : 0.f;
        if (!some) {
          m = fmaxf(top - lift, kNoScore);
          l = 0.f;
        } else if (__any_sync(0xffffffffu, mine && top > m + kLazy)) {
          // (rows without a query hold anything: they must not count)
          const float to = top > m + kLazy ? top - lift : m, al = ex2(m - to);
          m = to;
          l *= al;
          idle_wait(S, a, &S.pv_done[q], (ns - 1) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {  // (rare: few registers beside S matter more than speed)
            uint32_t r[8];
            tmem_ld8(o_tmem + 64 * half + 8 * c, r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * al);
            tmem_st8(o_tmem + 64 * half + 8 * c, r);
          }
        }
        const uint64_t neg = pack2(-m, -m), mul = pack2(f, f);
        uint64_t sum[2] = {0, 0};
        // P goes over this half's own scores, the first 32 tokens': the partner
        // and the second load are not disturbed
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 1) load(1);
          uint32_t p[kFp8 ? 1 : 16], hi[kFp8 ? 8 : 1], lo[kFp8 ? 8 : 1];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t s2 = pack2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
            float p0, p1;
            unpack2(kFp8 ? fma2(s2, mul, neg) : add2(s2, neg), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum[j & 1] = add2(sum[j & 1], pack2(p0, p1));
            if constexpr (kFp8) {
              uint32_t h2, l2;
              split_e4m3(p0, p1, h2, l2);
              hi[j / 2] = j & 1 ? hi[j / 2] | h2 << 16 : h2;
              lo[j / 2] = j & 1 ? lo[j / 2] | l2 << 16 : l2;
            } else {
              p[j] = pack_bf16(p0, p1);
            }
          }
          if constexpr (kFp8) {  // four codes a column: hi, and 16 columns further lo
            tmem_st8(s_tmem + 64 * half + 8 * c, hi);
            tmem_st8(s_tmem + 64 * half + 16 + 8 * c, lo);
          } else {
            tmem_st16(s_tmem + 64 * half + 16 * c, p);
          }
          if (c == 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_half[q]);
          }
        }
        float x[4];
        unpack2(sum[0], x[0], x[1]);
        unpack2(sum[1], x[2], x[3]);
        l += ((x[0] + x[1]) + (x[2] + x[3])) + (bad ? NAN : 0.f);
        tmem_wait_st();
      } else if (lane == 0) {
        mbar_arrive(&S.p_half[q]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[q]);
      some = true;
      ++ns;
    }
  } while ((step = w.next()));
  record();
}

// A programmatic dependent of the append launch, which itself starts its
// dependents only once everything before it is complete: the plan, q and the
// records' memory may be used at once, and only the trees' tiles wait for the
// launch before (the producer).  Every CTA waits for it before it ends, so
// that whoever follows this grid follows the append too.
template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  TcSmem<kFp8> &S = *reinterpret_cast<TcSmem<kFp8> *>(smem_raw);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (the grid is at most ctas_max: the record is there, whatever it holds)
  const TreeCta c = tree_at<TreeCta>(a, a.L.ctas)[blockIdx.x];
  const TreeHeader &hdr = *tree_at<const TreeHeader>(a, a.L.hdr);
  const bool ok = tree_plan_ok(a);
  if (!ok || static_cast<int>(blockIdx.x) >= hdr.n_ctas) {
    if (!ok && tid == 0) flag_error(reinterpret_cast<int32_t *>(a.ws), HW_DEV_BAD_PLAN);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  Walk w = {a, hdr.streams, c.head, c.group, c.span, c.tile, c.n_units, c.g, c.sp, 0,
            Ring<kFp8>::kStages + (c.wide ? 0 : Ring<kFp8>::kMore), !kFp8 && !c.wide, smem_u32(c.wide ? S.kv[0] : S.q[1])};
  w.begin();
  if (tid == 0) {
    for (int s = 0; s < TcSmem<kFp8>::kAll; ++s) {
      mbar_init(&S.kv_full[s], 1);
      mbar_init(&S.kv_empty[s], 2);  // one arrival a stream
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&S.q_full[q], 8);
      mbar_init(&S.s_full[q], 1);
      mbar_init(&S.p_half[q], 8);
      mbar_init(&S.p_full[q], 8);
      mbar_init(&S.pv_done[q], 1);
      mbar_init(&S.o_empty[q], 8);
      mbar_init(&S.scanned[q][0], 8);
      mbar_init(&S.scanned[q][1], 8);
    }
    mbar_init(&S.q_free, 2);
    mbar_init(&S.order, 1);
    mbar_init(&S.mma_done, 2);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&S.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, S.tmem, 0);
  if (warp == kWarpTma) {
    if ((tid & 31) == 0) producer(a, S, &tk, &tv, w);
  } else if (warp >= kWarpMma) {
    mma_issuer(a, S, tmem, w, warp - kWarpMma);
  } else {
    softmax(a, S, tmem, w, warp >> 3);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

namespace {
template <bool kFp8>
cudaError_t launch(const TreeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
  const size_t smem = sizeof(TcSmem<kFp8>);
  static bool configured = false;
  if (!configured) {
    const cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    configured = true;
  }
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
  return cudaLaunchKernelEx(&cfg, tree_tc_kernel<kFp8>, a, tk, tv);
}
}  // namespace

cudaError_t launch_tree_tc(const TreeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
  return a.dtype == HW_FP8_E4M3 ? launch<true>(a, tk, tv, s) : launch<false>(a, tk, tv, s);
}

}  // namespace hw
