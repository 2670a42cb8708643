// block_move.cu - token ranges moved within their pools (hw_block_move): blocks
// copied and forked, and slid together when freed ones lie between them.
//
//   pool[r][dst_m + j] = pool[r][src_m + j],  j < n_m,  for moves m = 0, 1, .. in this order
//   (K and V; r = layer, kv head; 4-bit caches: their scales too)
//
// Bound by DRAM: nothing is computed, and every byte should go once in and once out.  The
// bytes never pass through registers: one thread of a CTA has bulk copies bring
// chunks of 16 KB into a ring in shared memory and others take them out again, up to
// kStages - 2 chunks ahead, so a CTA keeps 64 KB on the way and two fit an SM.  Measured: 512
// bf16 tokens of 64 layers copied to three places (537 MB) 99 us, 5.4 TB/s; 1.8 GB of E4M3 blocks slid together
// 275 us, 6.6 TB/s.
//
// Moves that touch nothing of one another or of themselves (copies, forks) are cut into
// chunks for all CTAs.  Others are done row by row, a row's chunks in order by one
// CTA (a model's layers x heads x 2 are rows enough), and what keeps them right is:
//  - a move down goes from its first token up, a move up from its last one down: what a
//    chunk's store overwrites has then been read, by it or by a chunk before it, because
//    a chunk is stored only after its own load and those before it have landed, and the
//    loads under way behind it are of chunks that its destination does not meet;
//  - a move whose source or destination meets an earlier destination waits
//    (`drain`, found on the host) until all stores before it are written.
#include "hw_cache.h"
#include "hw_device.cuh"
#include "hw_sm100.cuh"

namespace hw {

using namespace sm100;

namespace {

__device__ int32_t g_move_flags;  // HW_DEV_* bits of the device's moves (hw_block_move_status)

constexpr int kThreads = 128;
constexpr int kStages = 6;
constexpr int kAhead = kStages - 2;  // chunks loaded ahead: a stage's store has two chunks' time to be read
constexpr uint32_t kChunk = 16384;
constexpr uint32_t kSmem = kStages * kChunk + 128;

__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Chunk after chunk of the CTA's work, in order: independent moves' chunks from the
// CTA's index on, every grid-th of all rows', else the chunks of a row, and
// then of the CTA's next row.
struct Walk {
  const MoveArgs &a;
  int per;         // tokens a chunk
  int64_t at;      // ordered: the row; else the index among a row's chunks and rows (at = row * in_row + chunk)
  int64_t in_row;  // chunks of a row (independent moves)
  int64_t end, step;
  int m, k, of;  // move, its chunk, its number of chunks
  __device__ __forceinline__ int chunks(int i) const { return (a.n[i] + per - 1) / per; }
  __device__ Walk(const MoveArgs &a_, int64_t first, int64_t step_) : a(a_), per(kChunk / a_.row_bytes), step(step_) {
    at = first;
    in_row = 0;
    if (a.ordered) {
      end = 2ll * a.rows;
      m = -1;
      k = of = 0;
      if (at < end) next_move();
    } else {
      for (int i = 0; i < a.n_moves; ++i) in_row += chunks(i);
      end = 2 * in_row * a.rows;
      if (at < end) find();
    }
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ void find() {
    int64_t c = at % in_row;
    for (m = 0; c >= chunks(m); ++m) c -= chunks(m);
    k = static_cast<int>(c);
    of = chunks(m);
  }
  __device__ void next_move() {  // (on to the next row behind the last; some move has tokens)
    do {
      if (++m == a.n_moves) {
        m = 0;
        at += step;
        if (at >= end) return;
      }
      of = chunks(m);
    } while (of == 0);
    k = 0;
  }
  __device__ __forceinline__ void next() {
    if (!a.ordered) {
      at += step;
      if (at < end) find();
    } else if (++k == of) {
      next_move();
    }
  }
  // Whether the chunk has to wait until everything before it is written: the first
  // of a move that meets an earlier one's destination.  (Rows do not meet.)
  __device__ __forceinline__ bool drain() const { return a.ordered && k == 0 && (a.drain[m >> 5] >> (m & 31) & 1); }
  __device__ __forceinline__ void place(uint8_t *&src, uint8_t *&dst, uint32_t &bytes) const {
    const int64_t r2 = a.ordered ? at : at / in_row;  // the K rows, then the V rows
    const bool v = r2 >= a.rows;
    uint8_t *pool = a.pool[v] + (v ? r2 - a.rows : r2) * a.capacity * a.row_bytes;
    const int kk = a.ordered && a.dst[m] > a.src[m] ? of - 1 - k : k;
    const int first = kk * per, n = min(per, a.n[m] - first);
    src = pool + (static_cast<int64_t>(a.src[m]) + first) * a.row_bytes;
    dst = pool + (static_cast<int64_t>(a.dst[m]) + first) * a.row_bytes;
    bytes = static_cast<uint32_t>(n) * a.row_bytes;
  }
};

// The scales' rows (a word a token): by a whole CTA, a batch of loads, then its stores.
__device__ void move_scales(const MoveArgs &a, int row) {
  constexpr int kPer = 8, kBatch = kPer * kThreads;
  uint32_t *s = a.kv_scale + static_cast<int64_t>(row) * a.capacity;
  const int tid = threadIdx.x;
  for (int m = 0; m < a.n_moves; ++m) {
    const int n = a.n[m];
    const bool up = a.dst[m] > a.src[m];
    for (int64_t b = 0; b < n; b += kBatch) {
      const int64_t first = up ? max(n - b - kBatch, static_cast<int64_t>(0)) : b;
      const int cnt = static_cast<int>(min(static_cast<int64_t>(kBatch), n - b));
      uint32_t w[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (tid + j * kThreads < cnt) w[j] = s[a.src[m] + first + tid + j * kThreads];
      __syncthreads();  // (every load of the batch before its stores)
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (tid + j * kThreads < cnt) s[a.dst[m] + first + tid + j * kThreads] = w[j];
      __syncthreads();  // (and these before the next loads)
    }
  }
}

__global__ void __launch_bounds__(kThreads) move_kernel(const __grid_constant__ MoveArgs a, int bulk_ctas) {
  extern __shared__ uint8_t raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~static_cast<uintptr_t>(127));
  __shared__ alignas(8) uint64_t full[kStages];
  if (static_cast<int>(blockIdx.x) >= bulk_ctas) {
    for (int row = blockIdx.x - bulk_ctas; row < a.rows; row += gridDim.x - bulk_ctas) move_scales(a, row);
    return;
  }
  if (threadIdx.x != 0) return;
  for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
  fence_mbar_init();
  Walk ld(a, blockIdx.x, bulk_ctas), st(a, blockIdx.x, bulk_ctas);
  int64_t issued = 0, done = 0;
  while (st.more()) {
    while (ld.more() && issued < done + kAhead) {
      if (ld.drain()) {
        if (done < issued) break;  // the chunks before it first
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        asm volatile("fence.proxy.async;" ::: "memory");
      } else {
        // the stage's last store, chunk issued - kStages <= done - 3, has been read: two may be left
        asm volatile("cp.async.bulk.wait_group.read 2;" ::: "memory");
      }
      uint8_t *src, *dst;
      uint32_t bytes;
      ld.place(src, dst, bytes);
      const int s = static_cast<int>(issued % kStages);
      mbar_arrive_expect_tx(&full[s], bytes);
      bulk_g2s(ring + s * kChunk, src, bytes, &full[s]);
      ++issued;
      ld.next();
    }
    uint8_t *src, *dst;
    uint32_t bytes;
    st.place(src, dst, bytes);
    const int s = static_cast<int>(done % kStages);
    // (a load that does not land: nothing is stored from it, nothing waits on, and the caller can
    // ask for it)
    if (!mbar_wait(&full[s], static_cast<uint32_t>(done / kStages & 1))) {
      flag_error(&g_move_flags, HW_DEV_TIMEOUT);
      break;
    }
    bulk_s2g(dst, ring + s * kChunk, bytes);
    ++done;
    st.next();
  }
  for (; done < issued; ++done) mbar_wait(&full[done % kStages], static_cast<uint32_t>(done / kStages & 1));
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace

cudaError_t launch_move(const MoveArgs &a, cudaStream_t s) {
  const int sms = device_sm_count();
  const int64_t most = 2ll * (sms > 0 ? sms : 152);
  const int per = static_cast<int>(kChunk) / a.row_bytes;
  int64_t items = 2ll * a.rows;
  if (!a.ordered) {
    int64_t in_row = 0;
    for (int m = 0; m < a.n_moves; ++m) in_row += (a.n[m] + per - 1) / per;
    items *= in_row;
  }
  const int bulk = static_cast<int>(items < most ? items : most);
  const int scale_ctas = a.kv_scale ? static_cast<int>(a.rows < most ? a.rows : most) : 0;
  const cudaError_t e = cudaFuncSetAttribute(move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  move_kernel<<<bulk + scale_ctas, kThreads, kSmem, s>>>(a, bulk);
  return cudaGetLastError();
}

cudaError_t read_move_flags(int32_t *flags, cudaStream_t s) {
  const int32_t none = 0;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(flags, g_move_flags, sizeof *flags);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_move_flags, &none, sizeof none);
  return e;
}

}  // namespace hw
