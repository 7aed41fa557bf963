// Causal attention with a sliding window, a few first tokens that stay visible
// and a learned relative position bias by buckets, forward and backward, on the
// 5th-generation tensor cores (head width 64, bf16 operands, fp32 softmax).
//
// Query i of a sequence of n tokens sees key j when
//   j <= i  and  (i - j < window  or  j < sinks),
// and its score is s_ij = q_i . k_j / 8 + table[bucket(i - j)][head].  With
// P = softmax over the visible keys and O = P V, the backward pass is
//   dV = P^T dO,  dP = dO V^T,  D_i = sum_j P_ij dP_ij,  dS = P o (dP - D),
//   dQ = dS K / 8,  dK = dS^T Q / 8,  dtable[b] = sum of dS_ij over the pairs
//   with bucket(i - j) = b.
// heads / kv_heads consecutive query heads share a key/value head, whose dK and
// dV are the sums over them.
//
// A CTA per (128-query block, head, sequence) walks the key blocks that its
// queries see: the blocks of the window up to the diagonal, and, where the
// window has left the first block, one narrow block of the sinks' keys.  Work
// is therefore proportional to the visible pairs and not to the square of the
// length.  The products are tcgen05.mma with the accumulators in tensor memory;
// the row threads own their rows (a whole one each in the forward kernel, half of
// one in the backward kernel), warps of their own issue the products (one forward,
// two backward) and another one the copies.
//
// Scores are kept in the log2 domain: t = s * log2(e) / 8 + bias * log2(e), so
// that an exponential is one ex2.  The bias enters a tile in one of three ways,
// each warp's by itself: as a constant of the row where every row of the warp lies
// within one bucket; as one of two constants where the buckets are wider than the
// tile; else by distance, from a table in shared memory in which the rows of a
// warp read consecutive words.  Heads with large entries take a fourth (kBigBias).
//
// The backward pass uses no atomics, so its results are bit-reproducible:
//   prep    -lse log2(e) and -D of every (head, query), in rows for the dQ CTAs
//           and as matrix operands for the dK/dV CTAs; -inf in the place of
//           -lse log2(e) for padded rows and rows that see nothing, whose P is
//           then 0.
//   main    dQ CTAs (128 queries, 64-key blocks) and dK/dV CTAs (128 keys,
//           64-query blocks, one query head of the group after the other).
//           The pairs of the sinks with queries that have left the window far
//           behind are not worth a dK/dV tile of their own per query block
//           (128 rows for a few keys): the dQ CTA, which has their P and dS,
//           multiplies them with dO and Q as well and leaves the few rows as a
//           partial sum.
//   finish  adds the partial sums of the sinks' dK, dV and of dtable in a fixed
//           order.
// dtable needs D to fp32 accuracy, while the D of the prep kernel carries the
// bf16 rounding of O (relative 2^-9).  A dQ row sees all its keys, so it keeps
// sum dS and sum P by bucket; sum over all buckets of its dS is then the error
// of D, e = D_exact - D, and the exact contribution of bucket b is
// sum_b dS - e sum_b P.
//
// What is rounded to bf16, and why: P and dS, since the products that read them
// take bf16 operands (fp16 ones would have to be o, dO, Q and K as well, whose
// range they do not have), and o, dQ, dK, dV, the results.  Each costs at most
// 2^-9 of the value; maxima, sums, D, lse and dtable are fp32 and wider.
//
// Every mbarrier wait is bounded as in attention.cu.  The shared-memory tiles'
// layout is described in attention_tiles.cuh.
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "../../include/gpipe.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_util.cuh"

namespace gp {
namespace {

using namespace attn;

constexpr int kMaxBuckets = 64;
constexpr int kMaxDistance = 4096;
constexpr int kMaxSinks = 64;
constexpr int kFwdColumns = 128, kBwdColumns = 32;  // of a tile that one thread has
constexpr float kHidden = -1e30f;  // a table entry at or below it hides its bucket

// Scores and lse carry a row's bias, and P in the backward pass is the exponential
// of their difference, so what they are rounded by is an error of P: some six
// roundings of 2^-24 of the bias, 2^-13 at 256.  A row whose visible entries are all
// below -256, or one of them above 256, has the largest of them, its base, taken out
// of the exponent instead: t - base loses nothing whatever their size, and lse alone
// gets it back.
constexpr float kBigBias = 256.f;
__device__ __forceinline__ bool big_bias(float t) { return fabsf(t) > kBigBias && fabsf(t) < INFINITY; }

struct WindowArgs {
  int nseq, seq, heads, kv_heads, window, sinks;
  const int32_t* lens;  // valid tokens per sequence, or NULL: seq
  const float* table;   // [buckets][heads], or NULL
  int ranks;            // non-empty buckets, by rising distance (0: no bias)
  int last;             // first distance of the last of them
  int near[2];          // from it on buckets have as many distances as a row has columns: [0] 128, [1] 32
  int start[kMaxBuckets];  // (first distance << 8) | bucket of each
  __host__ __device__ int first(int rank) const { return start[rank] >> 8; }
  __device__ __forceinline__ float entry(int rank, int head) const {
    const float t = table[static_cast<int64_t>(start[rank] & 255) * heads + head];
    return t <= kHidden ? -INFINITY : t;
  }
};

__device__ __forceinline__ int seq_len(const WindowArgs& a, int b) {
  return a.lens ? max(0, min(a.lens[b], a.seq)) : a.seq;
}

// Row threads: one warpgroup in the forward kernel (a thread has a whole row of
// a tile, so a row's maximum needs no exchange), two in the backward one (a
// thread has half a row).  The issuers and the loader are warps of one more
// warpgroup, since registers are passed on by whole warpgroups:
//   forward   256 threads launched with 128 registers; the row threads go up to
//             208, the others down to 48 (128 x 208 + 128 x 48 = 256 x 128);
//   backward  384 launched with 80; up to 96, down to 48
//             (256 x 96 + 128 x 48 = 384 x 80).
constexpr int FWD_ROWS = 128, BWD_ROWS = 256;
constexpr int FWD_THREADS = FWD_ROWS + 128, BWD_THREADS = BWD_ROWS + 128;
constexpr int FWD_REGS = 128, BWD_REGS = 80;  // a thread at launch
static_assert(FWD_ROWS * 208 + 128 * 48 == FWD_THREADS * FWD_REGS && BWD_ROWS * 96 + 128 * 48 == BWD_THREADS * BWD_REGS,
              "what the row threads take is what the others give");

// The whole warp waits; the answer is the same in every lane.
__device__ __forceinline__ bool warp_await(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* abort) {
  return __all_sync(0xffffffffu, lane_await(bar, parity, err, code, abort));
}
// For the row threads, which carry on after a wait that gave up: what they then
// compute is wrong and reported as such, but they read and write where they
// would have, all later waits return at once, and no thread is left waiting for
// one that has gone.
struct RowWait {
  int* err;
  volatile int* abort;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
    (void)lane_await(bar, parity, err, DERR_ACC_WAIT, abort);
    __syncwarp();
  }
};

// One lane of a converged warp, always the same one.  Unlike a comparison with
// the lane number it tells the compiler that what depends on it runs once per
// warp, so the products' operands go to uniform registers directly.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
// The warp's number, known to be uniform.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }

// A matrix descriptor as its first k step's; the following steps add to the
// address field (16-byte units): 2 along a K-major row, 128 down an MN-major tile.
__device__ __forceinline__ uint64_t kdesc0(uint32_t tile) { return kdesc(tile, 0); }
__device__ __forceinline__ uint64_t mndesc0(uint32_t tile) { return mndesc(tile, 0); }
constexpr uint64_t kKStep = 2, kMnStep = 128;

// A barrier of the N row threads, all of which come to it whatever they waited for in vain.
template <int N>
__device__ __forceinline__ void rows_barrier() {
  asm volatile("bar.sync 3, %0;" ::"n"(N) : "memory");
}

// The bias of one head in shared memory, and the rank of a distance's bucket.
//   value[kLow + d], d = -kLow .. near + kHigh - 1: by distance, for warps along
//   some of whose rows the bucket changes near the diagonal; a negative distance
//   is masked, whatever is read for it.  Such a warp has 32 rows and up to 128
//   columns with a distance below `near`, so none of near + 158 on.
//   by_rank[k]: a bucket's value.  It is all a row needs that lies in one bucket,
//   and beyond `near`, where a row meets at most two of them.
//   rank[d], d = 0 .. last (rank_of clamps).
//   *big: whether the head has big entries.  Values are in the log2 domain where it
//   has none, and as the table has them where it has.
// A table of values for every distance would be 16 KB larger at 4096 and leave an
// SM one backward CTA instead of two: that of 2 x 4096 tokens, 16 heads, 32
// buckets up to 4096 and their gradient took 572 us instead of 355.
struct Bias {
  static constexpr int kLow = 128, kHigh = 160;
  float *value, *by_rank;
  uint8_t* rank;
  int* big;
  int near, last;
  static __host__ __device__ constexpr int value_words(int near) { return (kLow + near + kHigh + 3) & ~3; }
  static __host__ __device__ constexpr int rank_bytes(int last) { return (last + 16) & ~15; }
  static __host__ __device__ constexpr int bytes(int near, int last) {
    return (value_words(near) + kMaxBuckets) * 4 + rank_bytes(last);
  }
  __device__ __forceinline__ Bias(uint8_t* at, int* big_, int near_, int last_) : big(big_), near(near_), last(last_) {
    value = reinterpret_cast<float*>(at);
    by_rank = value + value_words(near);
    rank = reinterpret_cast<uint8_t*>(by_rank + kMaxBuckets);
  }

  __device__ __forceinline__ int rank_of(int d) const { return rank[max(0, min(d, last))]; }
  // By the N row threads: the ranks, once (the first head's values come after a barrier).
  template <int N>
  __device__ __forceinline__ void fill_ranks(const WindowArgs& a, int tid) {
    for (int k = tid >> 5; k < a.ranks; k += N / 32)
      for (int d = a.first(k) + (tid & 31), end = k + 1 < a.ranks ? a.first(k + 1) : last + 1; d < end; d += 32)
        rank[d] = static_cast<uint8_t>(k);
  }
  template <int N>
  __device__ __forceinline__ void fill(const WindowArgs& a, int head, int tid) {
    rows_barrier<N>();  // nobody reads the previous head's any more
    if (tid < kMaxBuckets) {  // two warps, each of which looks at all entries
      // (a tile of a head with big entries takes a path of its own, in code apart from the others')
      const float t = tid < a.ranks ? a.entry(tid, head) : 0.f, other = (tid ^ 32) < a.ranks ? a.entry(tid ^ 32, head) : 0.f;
      const bool any = __any_sync(0xffffffffu, big_bias(t) || big_bias(other));
      if (tid < a.ranks) by_rank[tid] = any ? t : t * kLog2e;
      if (tid == 0) *big = any;
    }
    rows_barrier<N>();
    for (int x = tid; x < kLow + near + kHigh; x += N) value[x] = by_rank[rank_of(x - kLow)];
    rows_barrier<N>();
  }
  // The base of query i's row: the largest entry that it sees, if that is big.  (Not
  // kept: only heads with big entries ask for it.)
  __device__ __forceinline__ float base(const WindowArgs& a, int i) const {
    float x = -INFINITY;
#pragma unroll 1
    for (int k = rank_of(min(i, a.window - 1)); k >= 0; --k) x = fmaxf(x, by_rank[k]);
    if (a.sinks > 0) {
#pragma unroll 1
      for (int k = rank_of(i), end = rank_of(i - a.sinks + 1); k >= end; --k) x = fmaxf(x, by_rank[k]);
    }
    return big_bias(x) ? x : 0.f;
  }
  // What distance d adds to a score (log2 domain) of a row with this base, in a head with big entries.
  __device__ __forceinline__ float without(float base, int d) const { return (by_rank[rank_of(d)] - base) * kLog2e; }
};

// Bits 0..x of a word (x < 0: none, x >= 31: all).
__device__ __forceinline__ uint32_t bits_to(int x) {
  return x < 0 ? 0u : (x >= 31 ? 0xffffffffu : (2u << x) - 1u);
}

// Hide the columns of v whose bit in `see` is not set.
__device__ __forceinline__ void hide32(float* v, uint32_t see) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!((see >> i) & 1u)) v[i] = -INFINITY;
}

__device__ __forceinline__ void take_registers_fwd() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;"); }
__device__ __forceinline__ void give_registers_fwd() { asm volatile("setmaxnreg.dec.sync.aligned.u32 48;"); }
__device__ __forceinline__ void take_registers_bwd() { asm volatile("setmaxnreg.inc.sync.aligned.u32 96;"); }
__device__ __forceinline__ void give_registers_bwd() { asm volatile("setmaxnreg.dec.sync.aligned.u32 48;"); }

// Zero rows [from, to) of a tile of 128-byte rows, by one warp, for the async proxy.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to, int lane) {
  for (int x = from * 8 + lane; x < to * 8; x += 32)
    *reinterpret_cast<uint4*>(tile + x * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// 32 fp32 TMEM columns of this thread's lane, times scale, as bf16 into row r of a
// swizzled tile (units u0..u0+3) for the tile store; zeros unless `keep`
// (whatever the accumulator holds then).
__device__ __forceinline__ void stage_row32(uint32_t taddr, uint8_t* tile, int r, int u0, float scale, bool keep) {
  float v[32];
  ld_row32(taddr, v);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = keep ? v[i] * scale : 0.f;
  st_row32_bf16(tile, r, u0, v);
}

// Send a staged tile of 128 rows out, once `threads` of the row threads (whole
// warps, barrier `id`) have written it; rows behind the sequence's last are cut
// off.  Every thread of them comes here, whatever it waited for in vain.
__device__ __forceinline__ void send_tile(const CUtensorMap* map, int x, int y, int z, const uint8_t* tile, int id,
                                          int threads, bool leader) {
  fence_proxy_async_smem();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
  if (leader) {
    tma_store_3d(map, x, y, z, tile);
    bulk_commit();
    bulk_wait_read_all();  // before the CTA's shared memory goes
  }
}

__device__ __forceinline__ void zero_row64(__nv_bfloat16* dst) {
#pragma unroll
  for (int u = 0; u < 8; ++u) *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(0u, 0u, 0u, 0u);
}

// A position in a ring of stages: stage, and the parity of its current use.
struct RingPos {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ bool misaligned(const uint8_t* sm, int* err) {
  if (!(reinterpret_cast<uintptr_t>(sm) & 1023u)) return false;  // the tiles' swizzle needs 1024-byte alignment
  if (threadIdx.x == 0) atomicExch(err, DERR_ALIGN);
  return true;
}

// An issuer's last act (one lane): none of its products may still be running when the CTA exits.
__device__ __forceinline__ void drain_products(uint64_t* bfin, int* err) {
  tc_commit(bfin);
  mbar_wait_bounded(bfin, 0, err, DERR_DRAIN_WAIT);
}
// The loader's (one lane): none of the last copies into a ring, `loaded` in all, may still be landing.
__device__ __forceinline__ void drain_copies(uint64_t* full, int loaded, int stages, int* err) {
  for (int t = max(0, loaded - stages); t < loaded; ++t)
    mbar_wait_bounded(&full[t % stages], (t / stages) & 1, err, DERR_DRAIN_WAIT);
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
// A CTA takes 128 queries of one head; two of them share an SM, so that one's
// set-up, waits and stores run during the other's work.  Warps 0-3 are the rows,
// warp 4 issues the products, warp 5 the copies: what an issuer does between two
// products is on the rows' way (a wait and a commit take some hundred cycles),
// so each has as little to do as possible.  Per key tile t:
//   issuer:  S = Q K_{t+1}^T as soon as the rows have read S of tile t -> commit
//            bs;  O += P V_t once the rows wrote P -> commit bo, empty[stage].
//   loader:  the tile after the ring's last into a stage once that is empty.
//   rows:    wait bs; read S; arrive bsc; bias, mask, maximum; wait for the
//            previous O product; write P; arrive bp.
// P goes through tensor memory: as an A operand there it costs the products no
// shared-memory reads (at head width 64 an O product with P in shared memory
// reads 6 KB for 32 cycles of tensor work, above the 128 B a cycle there is).
// A row's maximum is only moved when a tile exceeds it by 2^8: P is then at most
// 2^8, which neither bf16 nor the fp32 sums mind, and O is seldom rescaled.
// The ring has three stages of K | V (57 us at 16384 tokens, 8 heads over 2, a
// window of 1024; 59 us with two), two where the bias needs the room.
//
// Bound by the row threads: a tile is a chain of one load of 128 scores, their
// maximum, exponentials, sums and the store of P, with two such warps on each
// quarter of an SM.  At that size 57 us is 583 TFLOP/s; the quarters issue in
// 48 % of the cycles, the exponentials' unit is busy for 34 %, the tensor cores
// for 32 %.  Two threads a row (64 columns each, a maximum exchanged) and the
// bias in steps of 32 columns were slower (the latter 107 us to 104 us at 8192
// tokens, 16 heads, a window of 2048).  4 x 512 tokens, 16 heads, a window of
// 128: 10 us, of which the launch is most.
constexpr int FWD_RING = T128;
constexpr float kMaxStep = 8.f;
constexpr int fwd_smem(int stages, int bias_bytes) { return FWD_RING + stages * 2 * T128 + 256 + bias_bytes; }

template <bool BIAS>
__global__ void __launch_bounds__(FWD_THREADS, 2)
    attn_window_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap to,
                           const __grid_constant__ WindowArgs a, __nv_bfloat16* __restrict__ out,
                           float* __restrict__ lse, int* err) {
  constexpr int kStages = BIAS ? 2 : 3;
  extern __shared__ __align__(1024) uint8_t sm[];
  if (misaligned(sm, err)) return;
  uint8_t* sQ = sm;
  uint8_t* ring = sm + FWD_RING;  // stages of K | V
  uint64_t* bar = reinterpret_cast<uint64_t*>(ring + kStages * 2 * T128);
  uint64_t *full = bar, *empty = bar + 3, *bs = bar + 6, *bo = bar + 7, *bfin = bar + 8, *bq = bar + 9, *bsc = bar + 10,
           *bp = bar + 11;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 12);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  uint8_t* rest = reinterpret_cast<uint8_t*>(bar) + 256;
  Bias bias(rest, reinterpret_cast<int*>(tslot + 2), a.near[0], a.last);

  const int tid = threadIdx.x, warp = warp_number(), ln = tid & 31;
  const int nqb = (a.seq + 127) / 128;
  // heads fastest, then sequences, then query blocks from the last (the longest rows first)
  const int h = static_cast<int>(blockIdx.x) % a.heads;
  const int lin = static_cast<int>(blockIdx.x) / a.heads;
  const int b = lin % a.nseq;
  const int qb = nqb - 1 - lin / a.nseq;
  const int q0 = qb * 128;
  const int64_t row0 = static_cast<int64_t>(b) * a.seq;
  const int D = a.heads * HD;
  const int kcol = D + (h / (a.heads / a.kv_heads)) * HD, vcol = kcol + a.kv_heads * HD;

  griddep_wait();
  const int n = seq_len(a, b);
  if (q0 >= n) {  // nothing but padding
    const int qi = q0 + tid;
    if (tid < FWD_ROWS && qi < a.seq) {
      zero_row64(out + (row0 + qi) * D + h * HD);
      lse[(row0 + qi) * a.heads + h] = -INFINITY;
    }
    return;
  }
  // key tiles: the sinks' (where the window has left it), then the window's up to the diagonal
  const int ws = max(0, q0 - a.window + 1) / 128;
  const int kt0 = a.sinks > 0 && ws > 0 ? 1 : 0;
  const int nt = kt0 + qb - ws + 1;
  auto tile_key = [&](int t) { return t < kt0 ? 0 : (ws + t - kt0) * 128; };
  auto width = [&](int t) {  // keys of a tile, in steps of 32
    return t < kt0 ? (a.sinks + 31) & ~31 : min(128, (n - tile_key(t) + 31) & ~31);
  };
  auto load_tile = [&](int t, int st) {
    uint8_t* dst = ring + st * 2 * T128;
    mbar_arrive_expect_tx(&full[st], 2 * T128);
    tma_load_3d(dst, &tq, kcol, tile_key(t), b, &full[st]);
    tma_load_3d(dst + T128, &tq, vcol, tile_key(t), b, &full[st]);
  };
  const int ahead = min(nt, kStages);
  if (tid == FWD_THREADS - 32) {  // the first copies leave before anything else is set up
    for (int i = 0; i < 10; ++i) mbar_init(&bar[i], 1);
    mbar_init(bsc, FWD_ROWS);
    mbar_init(bp, FWD_ROWS);
    *abort = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(bq, T128);
    tma_load_3d(sQ, &tq, h * HD, q0, b, bq);
    for (int t = 0; t < ahead; ++t) load_tile(t, t);
  }
  if (warp == 0) {
    tmem_alloc(tslot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // S at 0, O at 128, P (bf16) at 192

  if (warp >= FWD_ROWS / 32) {
    give_registers_fwd();
    if (warp == FWD_ROWS / 32 + 1) {  // ---- loader ----
      if (elect_one()) {
        RingPos lp;
        for (int i = 0; i < ahead; ++i) lp.next(kStages);
        int t = ahead;
        for (; t < nt; ++t) {
          if (!lane_await(&empty[lp.stage], lp.parity ^ 1u, err, DERR_TMA_WAIT, abort)) break;
          load_tile(t, lp.stage);
          lp.next(kStages);
        }
        // no copy may still be landing when the CTA exits
        drain_copies(full, t, kStages, err);
        mbar_wait_bounded(bq, 0, err, DERR_DRAIN_WAIT);
      }
      __syncwarp();
    } else if (warp == FWD_ROWS / 32) {  // ---- issuer: waits together, one lane issues ----
      constexpr uint32_t idO = mma_idesc_bf16(128, 64, false, true);
      const uint32_t tS = tmem, tO = tmem + 128, tP = tmem + 192;
      const uint64_t qd = kdesc0(smem_u32(sQ)), kd = kdesc0(smem_u32(ring)), vd = mndesc0(smem_u32(ring + T128));
      constexpr uint64_t kStage = 2 * T128 / 16;
      RingPos sp, op;  // of the next S, of the next O product
      auto issue_s = [&](int t) {
        const uint32_t idS = mma_idesc_bf16(128, width(t), false, false);
        const uint64_t k = kd + sp.stage * kStage;
        if (!warp_await(&full[sp.stage], sp.parity, err, DERR_MMA_WAIT, abort)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tS, qd + kk * kKStep, k + kk * kKStep, idS, kk ? 1u : 0u);
          tc_commit(bs);
        }
        sp.next(kStages);
        return true;
      };
      bool go = warp_await(bq, 0, err, DERR_MMA_WAIT, abort) && issue_s(0);
      for (int t = 0; t < nt && go; ++t) {
        if (t + 1 < nt) {  // the next S as soon as the rows have read this one
          go = warp_await(bsc, t & 1, err, DERR_MMA_WAIT, abort) && issue_s(t + 1);
          if (!go) break;
        }
        const int w = width(t), left = n - tile_key(t);
        if (left < w) {  // values behind the sequence's end: their P is 0, they themselves may be anything
          zero_rows(ring + op.stage * 2 * T128 + T128, left, w, ln);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t v = vd + op.stage * kStage;
        go = warp_await(bp, t & 1, err, DERR_MMA_WAIT, abort);  // P written, O rescaled
        if (!go) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (16 * kk < w) tc_mma_f16_ta(tO, tP + 8 * kk, v + kk * kMnStep, idO, (t | kk) ? 1u : 0u);
          tc_commit(bo);
          tc_commit(&empty[op.stage]);
        }
        op.next(kStages);
      }
      if (elect_one()) drain_products(bfin, err);
      __syncwarp();
    }
  } else {  // ---- rows ----
    take_registers_fwd();
    const uint32_t lane = static_cast<uint32_t>(warp * 32) << 16;
    const int qi = q0 + tid;
    const uint32_t tS = tmem + lane, tO = tmem + 128 + lane, tP = tmem + 192 + lane;
    const RowWait wait{err, abort};
    float m = -INFINITY, l = 0.f;
    if (BIAS) {
      bias.fill_ranks<FWD_ROWS>(a, tid);
      bias.fill<FWD_ROWS>(a, h, tid);
    }
    const bool big = BIAS && *bias.big;
    for (int t = 0; t < nt; ++t) {
      const int j0 = tile_key(t), w = width(t);
      const int d = qi - j0;  // distances d, d - 1, .. d - 127
      int rank = 0, other = 0;
      bool flat = true;
      if (BIAS) {
        rank = bias.rank_of(d);
        other = bias.rank_of(d - 127);
        flat = __all_sync(0xffffffffu, rank == other);
      }
      wait(bs, t & 1);
      tc_fence_after();
      float sv[128];
      {
        // columns behind the tile's width hold what was there before: the mask hides them
        const uint32_t at[4] = {tS, tS + 32, tS + 64, tS + 96};
        ld_rows<4>(at, sv);
      }
      tc_fence_before();
      mbar_arrive1(bsc);  // S may be overwritten by the next tile's product
      // scores = sc * s + cb (log2 domain): the raw scores with a bias that is the
      // same all along the row, or with the bias by distance already added
      float sc = kScaleLog2, cb = 0.f;
      if (BIAS) {
        if (__builtin_expect(big, 0)) {
          const float base = bias.base(a, qi);
#pragma unroll
          for (int i = 0; i < 128; ++i) sv[i] = fmaf(sv[i], kScaleLog2, bias.without(base, d - i));
          sc = 1.f;
        } else if (flat) {
          cb = bias.by_rank[rank];
        } else if (__all_sync(0xffffffffu, d - 127 >= bias.near)) {  // two buckets at most
          const float x = bias.by_rank[rank], y = bias.by_rank[other];
          const int first = d - a.first(rank);  // the column of the first bucket's first distance
#pragma unroll
          for (int i = 0; i < 128; ++i) sv[i] = fmaf(sv[i], kScaleLog2, i <= first ? x : y);
          sc = 1.f;
        } else {
          const float* at = bias.value + Bias::kLow + d;
#pragma unroll
          for (int i = 0; i < 128; ++i) sv[i] = fmaf(sv[i], kScaleLog2, at[-i]);
          sc = 1.f;
        }
      }
      if (__builtin_expect(w < 128 || !(j0 + 127 <= q0 && q0 + 127 - j0 < a.window), 0)) {  // some pair is hidden
        const int lo = d - a.window + 1, sk = a.sinks - j0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t see = bits_to(d - 32 * c) & (~bits_to(lo - 1 - 32 * c) | bits_to(sk - 1 - 32 * c));
          if (!__all_sync(0xffffffffu, see == 0xffffffffu)) hide32(sv + 32 * c, see);
        }
      }
      float mx8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
#pragma unroll
      for (int i = 0; i < 128; i += 2) mx8[(i >> 1) & 7] = fmax3(mx8[(i >> 1) & 7], sv[i], sv[i + 1]);
      const float mx = fmaf(
          fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7])), sc, cb);
      const float mn = mx > m + kMaxStep ? mx : m;  // (m = -inf: as soon as anything is visible)
      const float ms = mn == -INFINITY ? 0.f : mn;  // nothing visible yet: exp2(-inf - 0) = 0
      const float alpha = m == mn ? 1.f : ex2_approx(m - ms);
      m = mn;
      if (t > 0) {  // the previous O product reads P and writes O
        wait(bo, (t - 1) & 1);
        tc_fence_after();
      }
      const f32x2 sc2 = pack2(sc, sc), off2 = pack2(cb - ms, cb - ms);
      f32x2 rs[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (64 * c < w) {
          uint32_t u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float p0, p1;
            unpack2(fma2(pack2(sv[64 * c + 2 * i], sv[64 * c + 2 * i + 1]), sc2, off2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            rs[i & 3] = add2(rs[i & 3], pack2(p0, p1));
            u[i] = pack_bf16x2(p0, p1);
          }
          tmem_st32(tP + 32 * c, u);
        }
      }
      float r0, r1;
      unpack2(add2(add2(rs[0], rs[1]), add2(rs[2], rs[3])), r0, r1);
      if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {  // warp-uniform: tcgen05 loads/stores are per warp
        const f32x2 al2 = pack2(alpha, alpha);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t u[32];
          tmem_ld32(tO + 32 * c, u);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a0, a1;
            unpack2(mul2(pack2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), al2), a0, a1);
            u[i] = __float_as_uint(a0);
            u[i + 1] = __float_as_uint(a1);
          }
          tmem_st32(tO + 32 * c, u);
        }
      }
      tmem_st_wait();
      l = l * alpha + (r0 + r1);
      tc_fence_before();
      mbar_arrive1(bp);
    }
    wait(bo, (nt - 1) & 1);
    tc_fence_after();
    // l = 0: a row that sees nothing (padding, or every bucket of its keys hidden)
    const bool keep = qi < n && l != 0.f;
    stage_row32(tO, sQ, tid, 0, 1.0f / l, keep);  // in Q's place: its products are done
    stage_row32(tO + 32, sQ, tid, 4, 1.0f / l, keep);
    send_tile(&to, h * HD, q0, b, sQ, 1, FWD_ROWS, tid == 0);
    const float base = big ? bias.base(a, qi) : 0.f;
    if (qi < a.seq) lse[(row0 + qi) * a.heads + h] = keep ? fmaf(m + log2f(l), kLn2, base) : -INFINITY;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// Workspace, in this order (each part 256-byte aligned):
//   ld     float2 [nseq][heads][seqpad]: (-lse log2(e), -D) of every query, seqpad = seq rounded up to 128
//   terms  the same two as matrix operands, [nseq][heads][seqpad / 64][2][2 KB] (see kTerms)
//   far    float [nseq][heads][query blocks][sinks][128]: dV | dK of the sinks from one query block
//   base   float [nseq][kv_heads][sinks][128]: their dV | dK from the queries near them
//   tab    float [nseq][query blocks][heads][ranks]: dtable from one query block
struct WindowScratch {
  float2* ld;
  uint8_t* terms;
  float* far;   // NULL: no query block is far from the sinks
  float* base;
  float* tab;   // NULL: no table gradient
  size_t bytes;
};

__host__ __device__ constexpr int pad128(int x) { return (x + 127) / 128 * 128; }
// The first query block whose window has left the first key block.
__host__ __device__ constexpr int first_far_block(int window) { return (window + 254) / 128; }

// In the dK/dV CTAs a query is a column, and -lse and -D differ from column to
// column: added by the row threads they would be read from shared memory again by
// every row.  Instead the tensor cores add them, as one more k step of 16: A is 1
// in its first three columns and 0 in the others, B holds -8 lse (the score's
// scale is applied afterwards) or -D of the 64 queries in its first three columns,
// as a sum of three bf16 terms (24 bits).  Both are tiles without swizzle: 8 rows
// of 16 bytes (8 columns) follow each other, the two column halves are 128 bytes
// apart, the groups of 8 rows 256.  (The second column half is zeros, but for
// the mark of has_base; A is 0 there.)
constexpr int kTerms = 2048;       // bytes of B for 64 queries
constexpr int kOnes = 4096;        // of A
__device__ __forceinline__ uint64_t terms_desc(uint32_t tile) {
  return static_cast<uint64_t>((tile & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 16 |
         static_cast<uint64_t>(256 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}
// x as three bf16 terms, the rest of the 16 bytes zero (an infinity: in the first term).
__device__ __forceinline__ uint4 three_terms(float x) {
  const float hi = bf2f(f2bf(x)), r1 = isinf(hi) ? 0.f : x - hi;
  const float mid = bf2f(f2bf(r1)), lo = r1 - mid;
  return make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(lo, 0.f), 0u, 0u);
}

// Where the operands of query i are (the first of its two rows of 16 bytes).
__device__ __forceinline__ int64_t terms_at(const WindowArgs& a, int64_t b, int h, int i) {
  const int64_t at = (b * a.heads + h) * pad128(a.seq) + i;
  return (at >> 6) * (2 * kTerms) + (i >> 3 & 7) * 256 + (i & 7) * 16;
}
// Whether the row's -lse is without its base: said in the first column of the second
// half of the -lse operand, where A is 0.
__device__ __forceinline__ bool has_base(const uint8_t* terms, const WindowArgs& a, int64_t b, int h, int i) {
  return *reinterpret_cast<const uint16_t*>(terms + terms_at(a, b, h, i) + 128) != 0;
}

// Eight threads per (sequence, query, head) of the preparation, heads fastest.
struct PrepItem {
  int h, i;
  int64_t b;
  __device__ __forceinline__ explicit PrepItem(const WindowArgs& a) {
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
    const int seqpad = pad128(a.seq);
    h = static_cast<int>(item % a.heads);
    const int64_t bi = item / a.heads;
    i = static_cast<int>(bi % seqpad);
    b = bi / seqpad;
  }
};

// A row whose |lse| is above kBigLse and that has a base gets its -lse without the
// base.  lse has too few bits for the difference, so the row's sum is made again, by
// eight threads, each 8 columns.  (Below kBigLse lse itself is accurate enough, whatever the base.)
// 8192 tokens, 16 heads, a window of 2048, 32 buckets, forward and backward: 428 us, 643 with -1e9 in the
// first bucket, 6.3 ms with 1e4 added to all of them, which gives every row a base.
constexpr float kBigLse = 128.f;
__device__ __forceinline__ void take_out_base(const WindowArgs& a, const __nv_bfloat16* qkv, float2* ld, uint8_t* terms) {
  const PrepItem at(a);
  const int64_t b = at.b;
  const int h = at.h, i = at.i, sub = threadIdx.x & 7;
  const uint32_t eight = 0xffu << (threadIdx.x & 24);
  const int lo = max(0, i - a.window + 1), sinks = min(a.sinks, lo);  // keys 0 .. sinks - 1 and lo .. i
  float base = -INFINITY;
  for (int k = sub; k < a.ranks; k += 8) {
    const int from = a.first(k), to = k + 1 < a.ranks ? a.first(k + 1) : a.seq;  // distances from .. to - 1
    if (from <= i - lo || (sinks > 0 && from <= i && to > i - sinks + 1)) base = fmaxf(base, a.entry(k, h));
  }
#pragma unroll
  for (int s = 4; s > 0; s >>= 1) base = fmaxf(base, __shfl_xor_sync(eight, base, s));
  if (!big_bias(base)) return;
  const int64_t stride = static_cast<int64_t>(a.heads + 2 * a.kv_heads) * HD;
  const __nv_bfloat16* rows = qkv + b * a.seq * stride + 8 * sub;
  const __nv_bfloat16* keys = rows + (a.heads + h / (a.heads / a.kv_heads)) * HD;
  const uint4 q = *reinterpret_cast<const uint4*>(rows + i * stride + h * HD);
  // log2 sum_j 2^((s_ij - base) log2(e)) over the visible keys
  float m = -INFINITY, l = 0.f;
  int rank = a.ranks - 1;
  for (int x = 0; x < sinks + i - lo + 1; ++x) {
    const int j = x < sinks ? x : lo + x - sinks;
    while (a.first(rank) > i - j) --rank;  // (distances fall; the first bucket begins at 0)
    const uint4 k = *reinterpret_cast<const uint4*>(keys + j * stride);
    float s = 0.f;
    auto two = [&](uint32_t x, uint32_t y) {
      const float2 u = unpack_bf16x2(x), w = unpack_bf16x2(y);
      s = fmaf(u.y, w.y, fmaf(u.x, w.x, s));
    };
    two(q.x, k.x);
    two(q.y, k.y);
    two(q.z, k.z);
    two(q.w, k.w);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(eight, s, o);
    s = fmaf(s, kScaleLog2, (a.entry(rank, h) - base) * kLog2e);
    if (s > m) {
      l *= ex2_approx(m == -INFINITY ? m : m - s);
      m = s;
    }
    l += ex2_approx(m == -INFINITY ? s : s - m);
  }
  const float L = -(m + log2f(l));
  uint8_t* to = terms + terms_at(a, b, h, i);
  if (sub == 4) ld[(b * a.heads + h) * pad128(a.seq) + i].x = L;  // (each word by the thread that wrote it before)
  if (sub == 0) *reinterpret_cast<uint4*>(to) = three_terms(L * (1.f / kScaleLog2));
  if (sub == 1) *reinterpret_cast<uint4*>(to + 128) = make_uint4(1u, 0u, 0u, 0u);
}

// Bound by memory and its latency: reads o and dout, writes 72 bytes a (head, query),
// of which 64 are the two operands.  8192 tokens, 16 heads: 10.6 us for 43 MB (4.1
// TB/s, 60 % of the copy bandwidth).
template <bool TABLE>
__global__ void __launch_bounds__(256, 8) attn_window_prep_kernel(const __grid_constant__ WindowArgs a,
                                                                  const __nv_bfloat16* __restrict__ qkv,
                                                                  const __nv_bfloat16* __restrict__ o,
                                                                  const __nv_bfloat16* __restrict__ dout,
                                                                  const float* __restrict__ lse, float2* __restrict__ ld,
                                                                  uint8_t* __restrict__ terms) {
  griddep_wait();
  const PrepItem of(a);
  const int h = of.h, i = of.i, sub = threadIdx.x & 7, seqpad = pad128(a.seq);  // sub: 8 of the 64 columns
  const int64_t b = of.b;
  const bool in = b < a.nseq;
  const bool live = in && i < seq_len(a, static_cast<int>(in ? b : 0));
  float d = 0.f, v = -INFINITY;  // lse
  if (live) {
    const int64_t row = (b * a.seq + i) * a.heads + h;
    float x[8], y[8];
    load8(o + row * HD + 8 * sub, x);
    load8(dout + row * HD + 8 * sub, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) d = fmaf(x[e], y[e], d);
    v = lse[row];
  }
  float L = v == -INFINITY ? v : -v * kLog2e;  // a row that sees nothing: P = 0
#pragma unroll
  for (int s = 4; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
  griddep_launch();  // nothing but stores is left, so the main kernel's CTAs take no room for long before they run
  if (!in) return;
  const int64_t at = (b * a.heads + h) * seqpad + i;
  if (sub == 4) ld[at] = make_float2(L, -d);
  if (sub < 4) {  // the two column halves of both
    uint8_t* tile = terms + (at >> 6) * (2 * kTerms) + (sub >> 1) * kTerms;
    const float x = sub & 2 ? -d : L * (1.f / kScaleLog2);
    *reinterpret_cast<uint4*>(tile + (i >> 3 & 7) * 256 + (sub & 1) * 128 + (i & 7) * 16) =
        sub & 1 ? make_uint4(0u, 0u, 0u, 0u) : three_terms(x);
  }
  if (TABLE && fabsf(v) > kBigLse && v != -INFINITY) take_out_base(a, qkv, ld, terms);
}

// Both kinds of CTA own 128 rows and walk 64-wide tiles; two CTAs share an SM,
// so that one's set-up, waits and stores run during the other's work.  S and dP
// (or their transposes) take 64 tensor-memory columns each; warpgroup g of the
// two row warpgroups has columns 32 g .. 32 g + 31 of every row.
//   warp 8:  S, dP of tile t+1 as soon as the rows have read tile t's -> commit
//            bs.
//   warp 9:  the gradient products of tile t once the rows wrote P, dS ->
//            commit bo, and the ring's stage as empty.
//   warp 10: the copies; a tile into the ring once its stage is empty.
//   rows:    wait bs; read S, dP; arrive bsc; the elementwise gradient; wait
//            bo of tile t-1 (it reads P, dS); write them; arrive bp.
constexpr int BWD_ISSUER = BWD_ROWS / 32;  // the issuers' first warp
constexpr int DQ_V_STAGES = 2;
constexpr int BWD_BARS = 1024;  // the barriers come first, at addresses that take no registers
constexpr int kMaxSmem = 227 * 1024, kHalfSmem = 113 * 1024;  // of a CTA, and of each of two on an SM

struct BwdBars {
  uint64_t *full, *full2, *one, *bs, *bo, *bfin, *bsink, *bsd, *empty, *empty2, *bsc, *bp, *brow, *bq;
  uint32_t* tslot;
  volatile int* abort;
  int* big;
  __device__ __forceinline__ explicit BwdBars(uint8_t* at) {
    full = reinterpret_cast<uint64_t*>(at);
    full2 = full + 3;
    one = full + 5;   // the operands that stay for the whole walk
    bs = full + 6;
    bo = full + 7;
    bfin = full + 8;  // two
    bsink = full + 10;
    bsd = full + 11;
    empty = full + 12;
    empty2 = full + 15;
    bsc = full + 17;
    bp = full + 18;
    brow = full + 19;
    bq = full + 20;
    tslot = reinterpret_cast<uint32_t*>(full + 21);
    abort = reinterpret_cast<volatile int*>(tslot + 1);
    big = reinterpret_cast<int*>(tslot + 2);
  }
  // first(): the first copies, which leave before anything else is set up
  template <typename F>
  __device__ __forceinline__ uint32_t start(int warp, F&& first) const {
    if (threadIdx.x == BWD_THREADS - 32) {
      for (int i = 0; i < 17; ++i) mbar_init(&full[i], 1);
      for (int i = 17; i < 21; ++i) mbar_init(&full[i], BWD_ROWS);
      *abort = 0;
      fence_barrier_init();
      first();
    }
    if (warp == 0) {
      tmem_alloc(tslot, 256);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return *tslot;
  }
  __device__ __forceinline__ void finish(int warp, uint32_t tmem) const {
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
      tmem_dealloc(tmem, 256);
    }
  }
};

// Two predicated stores (a branch around them at every column costs more than they do).
__device__ __forceinline__ void store_if(uint32_t on, uint32_t at, float x, uint32_t at16, float x16) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b16 h;\n setp.ne.u32 p, %0, 0;\n cvt.rn.f16.f32 h, %4;\n"
      " @p st.shared.f32 [%1], %2;\n @p st.shared.b16 [%3], h;\n}\n" ::"r"(on),
      "r"(at), "f"(x), "r"(at16), "f"(x16)
      : "memory");
}

// Shared memory of a dQ CTA: barriers | dO | two value tiles | `stages` key
// tiles | bias | sums of the table's gradient | a Q tile for the sinks'
// products, in the place of the sums (which are done by then) where those are
// large enough.  Q itself is an A operand in tensor memory: the S product then
// reads 2 KB of shared memory for 32 cycles of tensor work instead of 6.
constexpr int DQ_DO = BWD_BARS, DQ_V = DQ_DO + T128, DQ_K = DQ_V + DQ_V_STAGES * T64;
constexpr int dq_sums(int ranks, int last) {
  return BWD_ROWS * 4 + (ranks + 1) * BWD_ROWS * 6 + (last / 32 + 1) * 4;
}
constexpr int dq_smem(int stages, int bias_bytes, int sums, bool far) {
  const int tile = T128 + 1024;  // with what its alignment may take
  return DQ_K + stages * T64 + bias_bytes + (far && sums < tile ? tile : sums);
}
// Shared memory of a dK/dV CTA: barriers | K | V | ones | `stages` of Q | dO |
// terms of -lse | terms of -D | bias.
constexpr int DKV_K = BWD_BARS, DKV_V = DKV_K + T128, DKV_ONES = DKV_V + T128, DKV_RING = DKV_ONES + kOnes,
              DKV_STAGE = 2 * T64 + 2 * kTerms;
constexpr int dkv_smem(int stages, int bias_bytes) {
  return DKV_RING + stages * DKV_STAGE + bias_bytes;
}

// MODE 0: no bias; 1: bias; 2: bias and its gradient.  WIDE: there are buckets beyond
// Bias::near besides the last one.
//
// dQ CTA: 128 queries, the window's 64-key tiles by rising key, the sinks' last.
// For the gradient of the table each row thread adds its dS and P by bucket into
// words of its own (no two threads share one).  Columns along which the bucket
// does not change add one sum.  Elsewhere the running sums are put down where a
// bucket ends: a bucket that begins and ends among the thread's columns is met
// nowhere else, so its sums are stored; only the first and the last are added to
// what is there.  Beyond the narrow buckets a row meets at most two, and adds each
// column to one of two sums: 2 x 4096 tokens, 16 heads, 32 buckets up to 4096 take
// 322 us instead of 353 (backward), 64 of them 541 instead of 594.  P's sums only
// weigh the error of D, which is some 2^-9 of dS: fp16 is enough for them, as sums
// of 2^14 P, whose 11 bits reach down to 2^-28 (a bucket that sums to less in a row
// keeps some of that row's error of D, 2^-9 of a gradient of that size).
//
// Bound by the row threads' instructions: some 2000 cycles a tile with the
// other CTA's work beside it, 4400 where the buckets change from column to
// column.  Figures of the whole backward pass are at its kernel.
constexpr float kSumP = 16384.f;
template <int MODE, bool WIDE>
__device__ void window_bwd_dq(const WindowArgs& a, const CUtensorMap* tq64, const CUtensorMap* tq128,
                              const CUtensorMap* td128, const CUtensorMap* tg, const WindowScratch& ws_,
                              const __nv_bfloat16* __restrict__ qkv, __nv_bfloat16* __restrict__ dqkv, int item,
                              int stages, int* err) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const BwdBars s(sm);
  uint8_t *sdO = sm + DQ_DO, *ringV = sm + DQ_V, *ringK = sm + DQ_K;
  uint8_t* rest = ringK + stages * T64;
  Bias bias(rest, s.big, a.near[1], a.last);
  if (MODE) rest += Bias::bytes(a.near[1], a.last);
  float* row_e = reinterpret_cast<float*>(rest);                               // [2][128]
  float* accS = row_e + BWD_ROWS;                                              // [ranks + 1][256]
  __half* accP = reinterpret_cast<__half*>(accS + (a.ranks + 1) * BWD_ROWS);   // [ranks + 1][256]
  uint32_t* ends = reinterpret_cast<uint32_t*>(accP + (a.ranks + 1) * BWD_ROWS);  // bit d: d is its bucket's first
  uint8_t* sinkQ = align1024(rest);

  const int tid = threadIdx.x, warp = warp_number(), ln = tid & 31;
  const int nqb = (a.seq + 127) / 128;
  const int h = item % a.heads;
  const int b = (item / a.heads) % a.nseq;
  const int qb = nqb - 1 - item / (a.heads * a.nseq);
  const int q0 = qb * 128;
  const int64_t row0 = static_cast<int64_t>(b) * a.seq;
  const int D = a.heads * HD;
  const int64_t ld = static_cast<int64_t>(a.heads + 2 * a.kv_heads) * HD;
  const int kcol = D + (h / (a.heads / a.kv_heads)) * HD, vcol = kcol + a.kv_heads * HD;

  griddep_wait();
  const int n = seq_len(a, b);
  float* tab = MODE == 2 ? ws_.tab + ((static_cast<int64_t>(b) * nqb + qb) * a.heads + h) * a.ranks : nullptr;
  if (q0 >= n) {  // a block of padding
    if (tid < 128 && q0 + tid < a.seq) zero_row64(dqkv + (row0 + q0 + tid) * ld + h * HD);
    if (MODE == 2 && tid < a.ranks) tab[tid] = 0.f;
    return;
  }
  const bool sink_tile = a.sinks > 0 && qb >= first_far_block(a.window);
  const int kt0 = a.sinks > 0 && !sink_tile ? 0 : max(0, q0 - a.window + 1) / 64;
  const int nwin = min(q0 + 127, n - 1) / 64 - kt0 + 1;
  const int nt = nwin + (sink_tile ? 1 : 0);
  auto tile_key = [&](int t) { return t < nwin ? (kt0 + t) * 64 : 0; };
  auto load_k = [&](int t, int stage) {
    mbar_arrive_expect_tx(&s.full[stage], T64);
    tma_load_3d(ringK + stage * T64, tq64, kcol, tile_key(t), b, &s.full[stage]);
  };
  auto load_v = [&](int t, int stage) {
    mbar_arrive_expect_tx(&s.full2[stage], T64);
    tma_load_3d(ringV + stage * T64, tq64, vcol, tile_key(t), b, &s.full2[stage]);
  };
  const int ahead = min(nt, DQ_V_STAGES);
  const uint32_t tmem = s.start(warp, [&] {
    mbar_arrive_expect_tx(s.one, T128);
    tma_load_3d(sdO, td128, h * HD, q0, b, s.one);
    for (int t = 0; t < ahead; ++t) {
      load_k(t, t);
      load_v(t, t);
    }
  });
  // S at 0, dP at 64, dQ at 128, dS (bf16) at 192, Q (bf16) at 224
  const uint32_t tS = tmem, tP = tmem + 64, tQ = tmem + 128, tdS = tmem + 192, tQa = tmem + 224;

  if (warp >= BWD_ISSUER) {
    give_registers_bwd();
    if (warp == BWD_ISSUER + 2) {  // ---- loader ----
      if (elect_one()) {
        RingPos kp, vp;
        for (int i = 0; i < ahead; ++i) {
          kp.next(stages);
          vp.next(DQ_V_STAGES);
        }
        int t = ahead;
        for (; t < nt; ++t) {
          if (t >= stages && !lane_await(&s.empty[kp.stage], kp.parity ^ 1u, err, DERR_TMA_WAIT, s.abort)) break;
          if (!lane_await(&s.empty2[vp.stage], vp.parity ^ 1u, err, DERR_TMA_WAIT, s.abort)) break;
          load_k(t, kp.stage);
          load_v(t, vp.stage);
          kp.next(stages);
          vp.next(DQ_V_STAGES);
        }
        drain_copies(s.full, t, stages, err);
        drain_copies(s.full2, t, DQ_V_STAGES, err);
        mbar_wait_bounded(s.one, 0, err, DERR_DRAIN_WAIT);
      }
      __syncwarp();
    } else if (warp == BWD_ISSUER) {  // ---- S = Q K_t^T, dP = dO V_t^T ----
      constexpr uint32_t id = mma_idesc_bf16(128, 64, false, false);
      bool go = warp_await(s.one, 0, err, DERR_MMA_WAIT, s.abort) && warp_await(s.bq, 0, err, DERR_MMA_WAIT, s.abort);
      if (go && n - q0 < 128) {  // padded queries: with Q = dO = 0 and P = 0 they add nothing to the sinks' sums
        zero_rows(sdO, n - q0, 128, ln);
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint64_t dO = kdesc0(smem_u32(sdO)), kd = kdesc0(smem_u32(ringK)), vd = kdesc0(smem_u32(ringV));
      RingPos kp, vp;
      for (int t = 0; t < nt && go; ++t) {
        go = warp_await(&s.full[kp.stage], kp.parity, err, DERR_MMA_WAIT, s.abort) &&
             warp_await(&s.full2[vp.stage], vp.parity, err, DERR_MMA_WAIT, s.abort);
        const int left = n - tile_key(t);
        if (go && left < 64) {  // keys behind the sequence's end: P = dS = 0, the rows themselves may be anything
          zero_rows(ringK + kp.stage * T64, left, 64, ln);
          zero_rows(ringV + vp.stage * T64, left, 64, ln);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t k = kd + kp.stage * (T64 / 16), v = vd + vp.stage * (T64 / 16);
        if (t > 0) go = go && warp_await(s.bsc, (t - 1) & 1, err, DERR_MMA_WAIT, s.abort);  // tile t-1's read out
        if (!go) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma_f16_ta(tS, tQa + 8 * kk, k + kk * kKStep, id, kk ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tP, dO + kk * kKStep, v + kk * kKStep, id, kk ? 1u : 0u);
          tc_commit(s.bs);
          tc_commit(&s.empty2[vp.stage]);
        }
        kp.next(stages);
        vp.next(DQ_V_STAGES);
      }
      if (elect_one()) drain_products(&s.bfin[0], err);
      __syncwarp();
    } else if (warp == BWD_ISSUER + 1) {  // ---- dQ += dS K_t ----
      constexpr uint32_t idQ = mma_idesc_bf16(128, 64, false, true);
      constexpr uint32_t idT = mma_idesc_bf16(128, 64, true, true);
      const uint64_t kd = mndesc0(smem_u32(ringK));
      RingPos gp_;
      bool go = true;
      for (int t = 0; t < nt; ++t) {
        const uint64_t k = kd + gp_.stage * (T64 / 16);
        go = warp_await(s.bp, t & 1, err, DERR_MMA_WAIT, s.abort);  // dS_t written
        if (!go) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma_f16_ta(tQ, tdS + 8 * kk, k + kk * kMnStep, idQ, (t | kk) ? 1u : 0u);
          tc_commit(s.bo);
          tc_commit(&s.empty[gp_.stage]);
        }
        gp_.next(stages);
      }
      if (sink_tile && go) {
        // The sinks' dV = P^T dO and dK = dS^T Q over this block's queries, in the columns of S and dP:
        // P (in the value tiles' place) and dS (in the key tiles') read MN-major.  Rows 64..127 of the
        // products come from the addresses 1024 bytes further (inside the CTA's shared memory) and are
        // not read.  Q comes once more, as a tile.
        go = warp_await(s.brow, 0, err, DERR_MMA_WAIT, s.abort);  // P, dS written, the table's sums done with
        if (go) {
          if (elect_one()) {
            mbar_arrive_expect_tx(s.bsink, T128);
            tma_load_3d(sinkQ, tq128, h * HD, q0, b, s.bsink);
          }
          __syncwarp();
          go = warp_await(s.bsink, 0, err, DERR_MMA_WAIT, s.abort);
        }
        if (go) {
          if (n - q0 < 128) {
            zero_rows(sinkQ, n - q0, 128, ln);
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t p = smem_u32(ringV), ds = smem_u32(ringK), q = smem_u32(sinkQ), dO = smem_u32(sdO);
#pragma unroll 1
            for (int kk = 0; kk < 8; ++kk) {
              tc_mma_f16(tS, sw128_desc(p + kk * 2048, 1024, 1024), mndesc(dO, kk), idT, kk ? 1u : 0u);
              tc_mma_f16(tP, sw128_desc(ds + kk * 2048, 1024, 1024), mndesc(q, kk), idT, kk ? 1u : 0u);
            }
            tc_commit(s.bsd);
          }
        }
      }
      if (elect_one()) drain_products(&s.bfin[1], err);
      __syncwarp();
    }
  } else {  // ---- rows ----
    take_registers_bwd();
    const int g = warp >> 2, r = tid & 127, qi = q0 + r;
    const uint32_t lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const RowWait wait{err, s.abort};
    {  // Q into tensor memory: half a row a thread, zeros for padded rows
      uint32_t u[16];
      const uint4* src = reinterpret_cast<const uint4*>(qkv + (row0 + min(qi, n - 1)) * ld + h * HD + 32 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = qi < n ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        u[4 * i] = x.x;
        u[4 * i + 1] = x.y;
        u[4 * i + 2] = x.z;
        u[4 * i + 3] = x.w;
      }
      tmem_st16(tQa + lane + 16 * g, u);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive1(s.bq);
    }
    const int nend = a.last / 32 + 1;
    float farS = 0.f, farP = 0.f;  // the last bucket's sums
    float rowS = 0.f;              // all of this thread's dS
    if (MODE == 2) {
      for (int k = 0; k < a.ranks; ++k) {
        accS[k * BWD_ROWS + tid] = 0.f;
        accP[k * BWD_ROWS + tid] = __float2half(0.f);
      }
      for (int x = tid; x < nend; x += BWD_ROWS) {
        uint32_t w = 0u;
        for (int k = 0; k < a.ranks; ++k)
          if (a.first(k) >> 5 == x) w |= 1u << (a.first(k) & 31);
        ends[x] = w;
      }
    }
    if (MODE) {
      bias.fill_ranks<BWD_ROWS>(a, tid);
      bias.fill<BWD_ROWS>(a, h, tid);
    }
    auto put = [&](int rank, float x, float p) {
      accS[rank * BWD_ROWS + tid] += x;
      __half* at = accP + rank * BWD_ROWS + tid;
      *at = __float2half(__half2float(*at) + p);
    };
    const float2 LD = ws_.ld[(static_cast<int64_t>(b) * a.heads + h) * pad128(a.seq) + qi];
    const f32x2 scale2 = pack2(kScaleLog2, kScaleLog2), D2 = pack2(LD.y, LD.y);
    auto tile = [&](auto big_head, float base, int t) {
      constexpr bool BIG = decltype(big_head)::value;
      const bool sink = t >= nwin;
      const int j0 = tile_key(t) + 32 * g;  // the key of this thread's column 0
      const int d = qi - j0;                // distances d, d - 1, .. d - 31
      int rank = 0;
      bool flat = true;
      if (MODE) {
        rank = bias.rank_of(d);
        flat = __all_sync(0xffffffffu, rank == bias.rank_of(d - 31));
      }
      // Two buckets at most: that of column 0 up to column last_of_first(), then that of distance d - 31.
      // (Asked for again where it is needed, which is cheaper than the registers to keep it in.)
      auto two = [&] { return WIDE && __all_sync(0xffffffffu, d - 31 >= bias.near); };
      auto last_of_first = [&] { return d - a.first(rank); };
      wait(s.bs, t & 1);
      tc_fence_after();
      float v[64];  // S (32 columns), then dP (32 columns), one round trip
      {
        const uint32_t at[2] = {tS + lane + 32 * g, tP + lane + 32 * g};
        ld_rows<2>(at, v);
      }
      tc_fence_before();
      mbar_arrive1(s.bsc);
      if (BIG) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], kScaleLog2, bias.without(base, d - i) + LD.x);
      } else if (MODE && !flat) {
        if (two()) {
          const float x = bias.by_rank[rank] + LD.x, y = bias.by_rank[bias.rank_of(d - 31)] + LD.x;
          const int first = last_of_first();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], kScaleLog2, i <= first ? x : y);
        } else {
          const float* at = bias.value + Bias::kLow + d;
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], kScaleLog2, at[-i] + LD.x);
        }
      } else {
        const float x = (MODE ? bias.by_rank[rank] : 0.f) + LD.x;
        const f32x2 x2 = pack2(x, x);
#pragma unroll
        for (int i = 0; i < 32; i += 2) unpack2(fma2(pack2(v[i], v[i + 1]), scale2, x2), v[i], v[i + 1]);
      }
      if (__builtin_expect(sink || !(j0 + 31 <= q0 && q0 + 127 - j0 < a.window), 0)) {
        const uint32_t window = sink ? 0u : ~bits_to(d - a.window);
        hide32(v, bits_to(d) & (window | bits_to(a.sinks - j0 - 1)));
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        v[i] = ex2_approx(v[i]);  // P
        v[i + 1] = ex2_approx(v[i + 1]);
        unpack2(mul2(pack2(v[i], v[i + 1]), add2(pack2(v[32 + i], v[33 + i]), D2)), v[32 + i], v[33 + i]);  // dS
      }
      if (MODE == 2) {
        f32x2 s2[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < 32; i += 2) s2[(i >> 1) & 1] = add2(s2[(i >> 1) & 1], pack2(v[32 + i], v[33 + i]));
        float x0, x1;
        unpack2(add2(s2[0], s2[1]), x0, x1);
        rowS += x0 + x1;
        if (flat) {
          f32x2 p2[2] = {0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 32; i += 2) p2[(i >> 1) & 1] = add2(p2[(i >> 1) & 1], pack2(v[i], v[i + 1]));
          float y0, y1;
          unpack2(add2(p2[0], p2[1]), y0, y1);
          if (__all_sync(0xffffffffu, rank == a.ranks - 1)) {
            farS += x0 + x1;
            farP += y0 + y1;
          } else {
            put(rank, x0 + x1, kSumP * (y0 + y1));
          }
        } else if (two()) {
          const int first = last_of_first(), other = bias.rank_of(d - 31);
          float s0 = 0.f, p0 = 0.f, s1 = 0.f, p1 = 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (i <= first) {
              s0 += v[32 + i];
              p0 = fmaf(v[i], kSumP, p0);
            } else {
              s1 += v[32 + i];
              p1 = fmaf(v[i], kSumP, p1);
            }
          }
          put(rank, s0, p0);
          if (other != rank) put(other, s1, p1);
        } else {
          // bit i: column i ends its bucket (its distance is the bucket's first).  From the bitmap,
          // distances low .. low + 31, the reverse of the columns' order.
          const int low = d - 31;
          const int wd = low >> 5;  // floor division
          const uint32_t w0 = wd >= 0 && wd < nend ? ends[wd] : 0u;
          const uint32_t w1 = wd + 1 >= 0 && wd + 1 < nend ? ends[wd + 1] : 0u;
          const uint32_t stop = __brev(__funnelshift_r(w0, w1, low & 31));
          float runS = 0.f, runP = 0.f;
          // the first bucket's sums wait in a spare word, the next ones go to their own
          uint32_t atS = smem_u32(accS + a.ranks * BWD_ROWS + tid), atP = smem_u32(accP + a.ranks * BWD_ROWS + tid);
          int step = (rank - 1 - a.ranks) * BWD_ROWS;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            runS += v[32 + i];
            runP = fmaf(v[i], kSumP, runP);
            const uint32_t ends_here = stop & (1u << i);
            store_if(ends_here, atS, runS, atP, runP);
            runS = ends_here ? 0.f : runS;
            runP = ends_here ? 0.f : runP;
            const int by = ends_here ? step : 0;
            step = ends_here ? -BWD_ROWS : step;
            atS += 4 * by;
            atP += 2 * by;
          }
          if (stop) put(rank, accS[a.ranks * BWD_ROWS + tid], __half2float(accP[a.ranks * BWD_ROWS + tid]));
          rank -= __popc(stop);
          if (rank >= 0) put(rank, runS, runP);  // (below 0: only columns behind the diagonal were left)
        }
      }
      uint32_t u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = pack_bf16x2(v[32 + 2 * i], v[33 + 2 * i]);
      if (t > 0) {  // the previous dQ product reads dS
        wait(s.bo, (t - 1) & 1);
        tc_fence_after();
      }
      tmem_st16(tdS + lane + 16 * g, u);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive1(s.bp);
      if (sink) {  // the last tile: its dP is there, so the value tiles' place is free; the key tiles' after dQ
        st_row32_bf16(ringV, r, 4 * g, v);
        wait(s.bo, t & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(ringK + swz(r, 4 * g + i)) =
              make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
      }
    };
    if (MODE && __builtin_expect(*bias.big, 0)) {
      const float base = has_base(ws_.terms, a, b, h, qi) ? bias.base(a, qi) : 0.f;
      for (int t = 0; t < nt; ++t) tile(std::bool_constant<MODE != 0>(), base, t);
    } else {
      for (int t = 0; t < nt; ++t) tile(std::false_type(), 0.f, t);
    }
    if (MODE == 2) {
      put(a.ranks - 1, farS, kSumP * farP);
      row_e[tid] = rowS;
      rows_barrier<BWD_ROWS>();
      // the error of D: a row's dS sum to it instead of 0 (a padded row's sums are 0 themselves)
      float e[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) e[c] = (row_e[32 * c + ln] + row_e[32 * c + ln + 128]) * (1.f / kSumP);
      for (int k = warp; k < a.ranks; k += BWD_ISSUER) {
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int at = k * BWD_ROWS + 32 * c + ln;
          x += accS[at] - e[c & 3] * __half2float(accP[at]);
        }
        x = warp_sum(x);
        if (ln == 0) tab[k] = x;
      }
    }
    if (sink_tile) {
      fence_proxy_async_smem();
      mbar_arrive1(s.brow);
      wait(s.bsd, 0);
      tc_fence_after();
      float* part = ws_.far + (((static_cast<int64_t>(b) * a.heads + h) * nqb + qb) * a.sinks + r) * 128 + 64 * g;
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // dV | dK
        float x[32];
        ld_row32((g ? tP : tS) + lane + 32 * c, x);
        if (r < a.sinks) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) store8(part + 32 * c + i, x + i);
        }
      }
    } else {
      wait(s.bo, (nt - 1) & 1);
      tc_fence_after();
    }
    stage_row32(tQ + lane + 32 * g, sdO, r, 4 * g, 0.125f, qi < n);  // in dO's place: its products are done
    send_tile(tg, h * HD, q0, b, sdO, 1, BWD_ROWS, tid == 0);
  }
  s.finish(warp, tmem);
}

// dK/dV CTA of 128 keys of one key/value head: iterations t = 0 .. group * nq - 1
// over the 64-query blocks that see them, one query head after the other.  dV
// and dK fill what S^T and dP^T leave of the CTA's half of the tensor memory, so
// P^T and dS^T take the place of S^T and dP^T, and the next S^T and dP^T follow
// the products that read them.  Each of the four has its own hand-off, so that
// dV += P^T dO and the next S^T run while the rows make dS^T, and dK += dS^T Q
// and the next dP^T while they make P^T.
// (With P^T and dS^T in shared memory instead, the products' reads of them and the
// rows' writes kept it busy, and a tile took 1.6 times as long.)
//
// Bound by the latency of that chain of four hand-offs, with the other CTA's to
// fill it.  The heads of a group follow each other in one CTA, which needs no partial
// sums of dK and dV; with few key blocks and a large group that leaves SMs idle.
template <int MODE, bool WIDE>
__device__ void window_bwd_dkv(const WindowArgs& a, const CUtensorMap* tq64, const CUtensorMap* tq128,
                               const CUtensorMap* td64, const CUtensorMap* tg, const WindowScratch& ws_,
                               __nv_bfloat16* __restrict__ dqkv, int item, int stages, int* err) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const BwdBars s(sm);
  uint8_t *sK = sm + DKV_K, *sV = sm + DKV_V, *ring = sm + DKV_RING;
  uint8_t* rest = ring + stages * DKV_STAGE;
  Bias bias(rest, s.big, a.near[1], a.last);

  const int tid = threadIdx.x, warp = warp_number(), ln = tid & 31;
  const int kvh = item % a.kv_heads;
  const int b = (item / a.kv_heads) % a.nseq;
  const int kb = item / (a.kv_heads * a.nseq);  // by rising key: in a full causal pass the longest first
  const int group = a.heads / a.kv_heads, h0 = kvh * group;
  const int k0 = kb * 128;
  const int64_t row0 = static_cast<int64_t>(b) * a.seq;
  const int D = a.heads * HD;
  const int64_t ld = static_cast<int64_t>(a.heads + 2 * a.kv_heads) * HD;
  const int kcol = D + kvh * HD, vcol = kcol + a.kv_heads * HD;
  const int seqpad = pad128(a.seq);

  griddep_wait();
  const int n = seq_len(a, b);
  if (k0 >= n) {  // a block of padding
    if (tid < 256 && k0 + (tid & 127) < a.seq)
      zero_row64(dqkv + (row0 + k0 + (tid & 127)) * ld + (tid < 128 ? kcol : vcol));
    return;
  }
  // the queries of this block: those whose window reaches it, and, for the sinks' block, the rest of
  // the 128-query blocks whose window reaches it (the dQ CTAs of the others account for the sinks)
  const int imax = min(n - 1, kb == 0 && a.sinks > 0 ? first_far_block(a.window) * 128 - 1 : k0 + 127 + a.window - 1);
  const int i0 = k0 / 64, nq = imax / 64 - i0 + 1;
  const int niter = group * nq;
  auto load_q = [&](int lh, int lq, int stage) {
    uint8_t* dst = ring + stage * DKV_STAGE;
    uint64_t* full = &s.full[stage];
    mbar_arrive_expect_tx(full, DKV_STAGE);
    tma_load_3d(dst, tq64, lh * HD, lq * 64, b, full);
    tma_load_3d(dst + T64, td64, lh * HD, lq * 64, b, full);
    bulk_load(dst + 2 * T64, ws_.terms + ((static_cast<int64_t>(b) * a.heads + lh) * (seqpad / 64) + lq) * (2 * kTerms),
              2 * kTerms, full);
  };
  const int ahead = min(niter, stages);
  const uint32_t tmem = s.start(warp, [&] {
    mbar_arrive_expect_tx(s.one, 2 * T128);
    tma_load_3d(sK, tq128, kcol, k0, b, s.one);
    tma_load_3d(sV, tq128, vcol, k0, b, s.one);
    for (int t = 0; t < ahead; ++t) load_q(h0 + t / nq, i0 + t % nq, t);
  });
  uint64_t *got_s = s.bs, *got_dp = s.bsd, *wrote_p = s.bp, *wrote_ds = s.bsc, *done_v = s.bo, *done_k = s.bsink;
  // S^T at 0, dP^T at 64, dV at 128, dK at 192; P^T and dS^T (bf16) over the columns of S^T and dP^T that
  // their thread has read: columns 0..31 of a tile at 0, columns 32..63 at 32
  const uint32_t tS = tmem, tdP = tmem + 64, tV = tmem + 128, tK = tmem + 192;

  if (warp >= BWD_ISSUER) {
    give_registers_bwd();
    if (warp == BWD_ISSUER + 2) {  // ---- loader ----
      if (elect_one()) {
        RingPos lp;
        for (int i = 0; i < ahead; ++i) lp.next(stages);
        int t = ahead, lh = h0 + t / nq, lq = i0 + t % nq;
        for (; t < niter; ++t) {
          if (!lane_await(&s.empty[lp.stage], lp.parity ^ 1u, err, DERR_TMA_WAIT, s.abort)) break;
          load_q(lh, lq, lp.stage);
          lp.next(stages);
          if (++lq == i0 + nq) {
            lq = i0;
            ++lh;
          }
        }
        drain_copies(s.full, t, stages, err);
        mbar_wait_bounded(s.one, 0, err, DERR_DRAIN_WAIT);
      }
      __syncwarp();
    } else if (warp == BWD_ISSUER) {  // ---- S^T = K Q_t^T, dP^T = V dO_t^T ----
      constexpr uint32_t idSP = mma_idesc_bf16(128, 64, false, false);
      const uint64_t k = kdesc0(smem_u32(sK)), v = kdesc0(smem_u32(sV)), qd = kdesc0(smem_u32(ring));
      RingPos sp;
      int qb = i0;
      const uint64_t ones = terms_desc(smem_u32(sm + DKV_ONES));
      bool go = warp_await(s.one, 0, err, DERR_MMA_WAIT, s.abort) && warp_await(s.bq, 0, err, DERR_MMA_WAIT, s.abort);
      for (int t = 0; t < niter && go; ++t) {
        go = warp_await(&s.full[sp.stage], sp.parity, err, DERR_MMA_WAIT, s.abort);
        const int left = n - qb * 64;
        if (left < 64) {  // padded queries: P = dS = 0, the rows themselves may be anything
          uint8_t* at = ring + sp.stage * DKV_STAGE;
          zero_rows(at, left, 64, ln);
          zero_rows(at + T64, left, 64, ln);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t q = qd + sp.stage * (DKV_STAGE / 16), dO = q + T64 / 16;
        const uint64_t tL = terms_desc(smem_u32(ring + sp.stage * DKV_STAGE + 2 * T64)), tD = tL + kTerms / 16;
        if (t > 0) go = go && warp_await(done_v, (t - 1) & 1, err, DERR_MMA_WAIT, s.abort);  // P^T of t-1 read
        if (!go) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tS, k + kk * kKStep, q + kk * kKStep, idSP, kk ? 1u : 0u);
          tc_mma_f16(tS, ones, tL, idSP, 1u);
          tc_commit(got_s);
        }
        if (t > 0 && !warp_await(done_k, (t - 1) & 1, err, DERR_MMA_WAIT, s.abort)) break;  // dS^T of t-1 read
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tdP, v + kk * kKStep, dO + kk * kKStep, idSP, kk ? 1u : 0u);
          tc_mma_f16(tdP, ones, tD, idSP, 1u);
          tc_commit(got_dp);
        }
        if (++qb == i0 + nq) qb = i0;
        sp.next(stages);
      }
      if (elect_one()) drain_products(&s.bfin[0], err);
      __syncwarp();
    } else if (warp == BWD_ISSUER + 1) {  // ---- dV += P^T dO_t, dK += dS^T Q_t ----
      constexpr uint32_t idKV = mma_idesc_bf16(128, 64, false, true);
      const uint64_t qd = mndesc0(smem_u32(ring));
      RingPos gp_;
      for (int t = 0; t < niter; ++t) {
        const uint64_t q = qd + gp_.stage * (DKV_STAGE / 16), dO = q + T64 / 16;
        if (!warp_await(wrote_p, t & 1, err, DERR_MMA_WAIT, s.abort)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16_ta(tV, tS + 32 * (kk >> 1) + 8 * (kk & 1), dO + kk * kMnStep, idKV, (t | kk) ? 1u : 0u);
          tc_commit(done_v);
        }
        if (!warp_await(wrote_ds, t & 1, err, DERR_MMA_WAIT, s.abort)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16_ta(tK, tdP + 32 * (kk >> 1) + 8 * (kk & 1), q + kk * kMnStep, idKV, (t | kk) ? 1u : 0u);
          tc_commit(done_k);
          tc_commit(&s.empty[gp_.stage]);
        }
        gp_.next(stages);
      }
      if (elect_one()) drain_products(&s.bfin[1], err);
      __syncwarp();
    }
  } else {  // ---- rows ----
    take_registers_bwd();
    const int g = warp >> 2, r = tid & 127, kr = k0 + r;
    const uint32_t lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const RowWait wait{err, s.abort};
    int hq = h0, qb = i0;
    {  // the ones: this thread's half of row r
      uint8_t* at = sm + DKV_ONES + (r >> 3) * 256 + g * 128 + (r & 7) * 16;
      *reinterpret_cast<uint4*>(at) =
          g ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(pack_bf16x2(1.f, 1.f), pack_bf16x2(1.f, 0.f), 0u, 0u);
      fence_proxy_async_smem();
      mbar_arrive1(s.bq);
    }
    const f32x2 scale2 = pack2(kScaleLog2, kScaleLog2);
    auto tile = [&](auto big_head, int t) {
      constexpr bool BIG = decltype(big_head)::value;
      const int q0 = qb * 64 + 32 * g;  // the query of this thread's column 0
      const int d = q0 - kr;            // distances d .. d + 31
      int rank = 0, other = 0;
      bool flat = true;
      if (MODE) {
        rank = bias.rank_of(d + 31);
        other = bias.rank_of(d);
        flat = __all_sync(0xffffffffu, rank == other);
      }
      wait(got_s, t & 1);
      tc_fence_after();
      float v[32];  // S^T - 8 lse
      ld_row32(tS + lane + 32 * g, v);
      if (BIG) {  // a column's base: lane q has column q's
        const float base = has_base(ws_.terms, a, b, hq, q0 + ln) ? bias.base(a, q0 + ln) : 0.f;
#pragma unroll
        for (int q = 0; q < 32; ++q)
          v[q] = fmaf(v[q], kScaleLog2, bias.without(__shfl_sync(0xffffffffu, base, q), d + q));
      } else if (MODE && !flat) {
        if (WIDE && __all_sync(0xffffffffu, d >= bias.near)) {  // two buckets at most
          const float x = bias.by_rank[rank], y = bias.by_rank[other];
          const int first = a.first(rank) - d;  // the column of the second bucket's first distance
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = fmaf(v[q], kScaleLog2, q >= first ? x : y);
        } else {
          const float* at = bias.value + Bias::kLow + d;
#pragma unroll
          for (int q = 0; q < 32; q += 2)
            unpack2(fma2(pack2(v[q], v[q + 1]), scale2, pack2(at[q], at[q + 1])), v[q], v[q + 1]);
        }
      } else if (MODE) {
        const float c = bias.by_rank[rank];
        const f32x2 c2 = pack2(c, c);
#pragma unroll
        for (int q = 0; q < 32; q += 2) unpack2(fma2(pack2(v[q], v[q + 1]), scale2, c2), v[q], v[q + 1]);
      } else {
#pragma unroll
        for (int q = 0; q < 32; q += 2) unpack2(mul2(pack2(v[q], v[q + 1]), scale2), v[q], v[q + 1]);
      }
      if (__builtin_expect(!(q0 >= k0 + 127 && q0 + 31 - k0 < a.window), 0))  // some pair may be hidden
        hide32(v, bits_to(kr < a.sinks ? 31 : a.window - 1 - d) & ~bits_to(-d - 1));
      uint32_t u[16];
#pragma unroll
      for (int q = 0; q < 32; q += 2) {
        v[q] = ex2_approx(v[q]);  // P^T
        v[q + 1] = ex2_approx(v[q + 1]);
        u[q / 2] = pack_bf16x2(v[q], v[q + 1]);
      }
      tmem_st16(tS + lane + 32 * g, u);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive1(wrote_p);
      wait(got_dp, t & 1);
      tc_fence_after();
      float w[32];  // dP^T - D
      ld_row32(tdP + lane + 32 * g, w);
#pragma unroll
      for (int q = 0; q < 32; q += 2) {
        float s0, s1;
        unpack2(mul2(pack2(v[q], v[q + 1]), pack2(w[q], w[q + 1])), s0, s1);  // dS^T
        u[q / 2] = pack_bf16x2(s0, s1);
      }
      tmem_st16(tdP + lane + 32 * g, u);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive1(wrote_ds);
    };
    if (MODE) {
      bias.fill_ranks<BWD_ROWS>(a, tid);
      for (int t = 0; t < niter; ++hq) {
        bias.fill<BWD_ROWS>(a, hq, tid);
        if (__builtin_expect(*bias.big, 0)) {
          for (qb = i0; qb < i0 + nq; ++qb, ++t) tile(std::bool_constant<MODE != 0>(), t);
        } else {
          for (qb = i0; qb < i0 + nq; ++qb, ++t) tile(std::false_type(), t);
        }
      }
    } else {
      for (int t = 0; t < niter; ++t) {
        tile(std::false_type(), t);
        if (++qb == i0 + nq) qb = i0;
      }
    }
    wait(done_v, (niter - 1) & 1);
    wait(done_k, (niter - 1) & 1);
    tc_fence_after();
    // warpgroup 0 stores dV, 1 dK, in the place of V and K, whose products are done.  Of the sinks'
    // rows the finish kernel makes the sum with the query blocks far from them.
    const uint32_t acc = (g ? tK : tV) + lane;
    uint8_t* tile_out = g ? sK : sV;
#pragma unroll
    for (int c = 0; c < 2; ++c) stage_row32(acc + 32 * c, tile_out, r, 4 * c, g ? 0.125f : 1.f, kr < n);
    send_tile(tg, g ? kcol : vcol, k0, b, tile_out, 1 + g, 128, r == 0);
    if (ws_.far && kb == 0) {  // dV | dK
      float* part = ws_.base + ((static_cast<int64_t>(b) * a.kv_heads + kvh) * a.sinks + r) * 128 + 64 * g;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x[32];
        ld_row32(acc + 32 * c, x);
        if (kr < a.sinks && kr < n) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) store8(part + 32 * c + i, x + i);
        }
      }
    }
  }
  s.finish(warp, tmem);
}

// One launch for both kinds, the dK/dV CTAs first (they have more to do).
// 2 x 4096 tokens, 16 heads, everything visible, 32 buckets with their gradient:
// 283 us (five products: 606 TFLOP/s); the quarters of an SM issue in 56 % of the
// cycles, the tensor cores are busy for 41 %, the exponentials' unit for 22 %.
// 8192 tokens, a window of 2048, 16 sinks, buckets up to 1024: 305 us.  4 x 512
// tokens, a window of 128, no table: 21 us.
// The row threads' 96 registers do not hold everything: the five forms spill (264 to
// 516 bytes of reloads in the code), and at 2 x 4096 tokens 2.4 % of the
// instructions are reloads, some seven a tile and warp.
template <int MODE, bool WIDE>
__global__ void __launch_bounds__(BWD_THREADS, 2)
    attn_window_bwd_kernel(const __grid_constant__ CUtensorMap tq64, const __grid_constant__ CUtensorMap tq128,
                           const __grid_constant__ CUtensorMap td64, const __grid_constant__ CUtensorMap td128,
                           const __grid_constant__ CUtensorMap tg, const __grid_constant__ WindowArgs a,
                           const __grid_constant__ WindowScratch ws_, const __nv_bfloat16* __restrict__ qkv,
                           __nv_bfloat16* __restrict__ dqkv, int n_dkv, int dkv_stages, int dq_stages, int* err) {
  extern __shared__ __align__(1024) uint8_t sm[];
  if (misaligned(sm, err)) return;
  const int x = static_cast<int>(blockIdx.x);
  if (x < n_dkv)
    window_bwd_dkv<MODE, WIDE>(a, &tq64, &tq128, &td64, &tg, ws_, dqkv, x, dkv_stages, err);
  else
    window_bwd_dq<MODE, WIDE>(a, &tq64, &tq128, &td128, &tg, ws_, qkv, dqkv, x - n_dkv, dq_stages, err);
}

// Blocks 0 .. n_sink-1: one sink key of one (sequence, key/value head); thread
// (slice, c) adds column c of its dV | dK over every fourth far query block, and
// the slices are added in order.  Blocks n_sink ..: dtable of one head; a warp
// adds every sixteenth (sequence, query block), lanes over the ranks, and the
// warps are added in order.  Bound by latency: 4 us for 4 sinks of 64 (sequence,
// head)s, 6.7 us for 16 sinks of 16 heads over 46 query blocks and the table.  (The
// last CTA of the main kernel to leave a partial sum adding them instead, by a
// counter, saved the launch and cost each CTA more: 393 us became 401 us for
// forward and backward of 2 x 4096 tokens.)
constexpr int kFinishThreads = 512;
__global__ void __launch_bounds__(kFinishThreads) attn_window_finish_kernel(const __grid_constant__ WindowArgs a,
                                                                            const __grid_constant__ WindowScratch ws_,
                                                                            __nv_bfloat16* __restrict__ dqkv,
                                                                            float* __restrict__ dtable, int n_sink) {
  griddep_wait();
  griddep_launch();
  __shared__ double part[kFinishThreads / 32][kMaxBuckets];
  __shared__ float slice_sum[4][128];
  const int nqb = (a.seq + 127) / 128, tid = threadIdx.x;
  const int x = static_cast<int>(blockIdx.x);
  if (x < n_sink) {
    const int c = tid & 127, slice = tid >> 7;
    const int j = x % a.sinks, kvh = (x / a.sinks) % a.kv_heads, b = x / (a.sinks * a.kv_heads);
    const int n = seq_len(a, b);
    if (j >= n) return;
    const int group = a.heads / a.kv_heads, D = a.heads * HD;
    float v = slice ? 0.f : ws_.base[((static_cast<int64_t>(b) * a.kv_heads + kvh) * a.sinks + j) * 128 + c];
    for (int g = 0; g < group; ++g) {
      const float* far = ws_.far + (static_cast<int64_t>(b) * a.heads + kvh * group + g) * nqb * a.sinks * 128;
#pragma unroll 8
      for (int qb = first_far_block(a.window) + slice; qb <= (n - 1) / 128; qb += 4)
        v += far[(static_cast<int64_t>(qb) * a.sinks + j) * 128 + c];
    }
    slice_sum[slice][c] = v;
    __syncthreads();
    if (slice) return;
    v = ((slice_sum[0][c] + slice_sum[1][c]) + slice_sum[2][c]) + slice_sum[3][c];
    const int64_t ld = static_cast<int64_t>(a.heads + 2 * a.kv_heads) * HD;
    __nv_bfloat16* dst = dqkv + (static_cast<int64_t>(b) * a.seq + j) * ld + D + kvh * HD;
    if (c < 64) dst[a.kv_heads * HD + c] = f2bf(v);
    else dst[c - 64] = f2bf(v * 0.125f);
    return;
  }
  const int h = x - n_sink, warp = tid >> 5, ln = tid & 31;
  const int64_t parts = static_cast<int64_t>(a.nseq) * nqb;
  for (int k = ln; k < a.ranks; k += 32) {
    double s = 0.0;
#pragma unroll 8
    for (int64_t p = warp; p < parts; p += kFinishThreads / 32) s += ws_.tab[(p * a.heads + h) * a.ranks + k];
    part[warp][k] = s;
  }
  __syncthreads();
  if (tid >= a.ranks) return;
  double s = 0.0;
  for (int w = 0; w < kFinishThreads / 32; ++w) s += part[w][tid];
  dtable[static_cast<int64_t>(a.start[tid] & 255) * a.heads + h] += static_cast<float>(s);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// bf16 tensor [nseq][seq][cols], boxes of 64 columns x box_rows rows of one
// sequence, 128-byte swizzle; rows behind a sequence's last are read as zeros.
bool make_tmap(CUtensorMap* m, const void* base, int64_t cols, int64_t seq, int64_t nseq, int box_rows) {
  EncodeFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(seq), static_cast<cuuint64_t>(nseq)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(cols) * seq * 2};
  cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// n^e >= md^k me^(e - k), in whole numbers of 32 words (e is at most 32, and 4096^32 has 385 bits).
bool power_at_least(int n, int e, int md, int k, int me) {
  uint32_t x[32] = {1}, y[32] = {1};
  auto times = [](uint32_t* v, uint32_t f) {
    uint64_t carry = 0;
    for (int i = 0; i < 32; ++i) {
      carry += static_cast<uint64_t>(v[i]) * f;
      v[i] = static_cast<uint32_t>(carry);
      carry >>= 32;
    }
  };
  for (int i = 0; i < e; ++i) {
    times(x, static_cast<uint32_t>(n));
    times(y, static_cast<uint32_t>(i < k ? md : me));
  }
  for (int i = 31; i >= 0; --i)
    if (x[i] != y[i]) return x[i] > y[i];
  return true;
}

int check_buckets(int buckets, int max_distance) {
  if (buckets < 2 || buckets > kMaxBuckets || max_distance <= buckets / 2 || max_distance > kMaxDistance)
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "position buckets: need 2 <= num_buckets <= %d and num_buckets / 2 < max_distance <= %d",
                     kMaxBuckets, kMaxDistance);
  return GPIPE_OK;
}

void bucket_starts(int buckets, int max_distance, int32_t* starts) {
  const int me = buckets / 2, m = buckets - me;
  for (int b = 0; b < me; ++b) starts[b] = b;
  for (int k = 0; k < m; ++k) {
    const double x = me * std::pow(static_cast<double>(max_distance) / me, static_cast<double>(k) / m);
    const double near = std::nearbyint(x);
    // pow is off by parts in 1e15; only next to a whole number does that decide
    if (std::fabs(x - near) > 1e-6)
      starts[me + k] = static_cast<int32_t>(std::ceil(x));
    else
      starts[me + k] = static_cast<int32_t>(near) + (power_at_least(static_cast<int>(near), m, max_distance, k, me) ? 0 : 1);
  }
}

int window_args(WindowArgs& a, int nseq, int seq, int heads, int kv_heads, int window, int sinks, const int32_t* lens,
                const float* table, int buckets, int max_distance) {
  if (nseq < 1 || seq < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads || heads > 4096)
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "attention_window: need nseq, seq >= 1 and heads (at most 4096) a multiple of kv_heads >= 1");
  if (static_cast<int64_t>(nseq) * seq > (int64_t(1) << 30))
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window: nseq * seq must be at most 2^30");
  if (window < 1 || sinks < 0 || sinks > kMaxSinks)
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window: need window >= 1 and 0 <= sinks <= %d", kMaxSinks);
  if (static_cast<int64_t>(nseq) * heads * ((seq + 127) / 128) > (int64_t(1) << 28))
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window: more than 2^28 blocks of 128 queries");
  a = WindowArgs{};
  a.nseq = nseq;
  a.seq = seq;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.window = window < seq ? window : seq;
  a.sinks = sinks < seq ? sinks : seq;
  a.lens = lens;
  if ((table != nullptr) != (buckets != 0))
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window: a bias table goes with num_buckets > 0, none with 0");
  if (!table) return GPIPE_OK;
  const int rc = check_buckets(buckets, max_distance);
  if (rc) return rc;
  a.table = table;
  int32_t starts[kMaxBuckets];
  bucket_starts(buckets, max_distance, starts);
  for (int b = 0; b < buckets; ++b) {
    // a bucket that begins where the next one does is empty, one that begins behind the longest distance unused
    if ((b + 1 < buckets && starts[b + 1] == starts[b]) || starts[b] >= seq) continue;
    a.start[a.ranks++] = starts[b] << 8 | b;
  }
  a.last = a.near[0] = a.near[1] = a.first(a.ranks - 1);
  for (int i = 0; i < 2; ++i)
    for (int k = a.ranks - 2; k >= 0 && a.first(k + 1) - a.first(k) >= (i ? kBwdColumns : kFwdColumns); --k)
      a.near[i] = a.first(k);
  return GPIPE_OK;
}

bool has_far(int seq, int window, int sinks) {
  return sinks > 0 && (seq + 127) / 128 > first_far_block(window < seq ? window : seq);
}

WindowScratch window_scratch(void* base, int nseq, int seq, int heads, int window, int sinks, int ranks) {
  WindowScratch w = {};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = static_cast<uint8_t*>(base) + off;
    off += (bytes + 255) & ~static_cast<size_t>(255);
    return p;
  };
  const size_t nqb = (static_cast<size_t>(seq) + 127) / 128, nh = static_cast<size_t>(nseq) * heads;
  w.ld = reinterpret_cast<float2*>(take(nh * nqb * 128 * sizeof(float2)));
  w.terms = take(nh * nqb * 4 * kTerms);
  if (has_far(seq, window, sinks)) {
    const size_t s = sinks < seq ? sinks : seq;
    w.far = reinterpret_cast<float*>(take(nh * nqb * s * 128 * sizeof(float)));
    w.base = reinterpret_cast<float*>(take(nh * s * 128 * sizeof(float)));
  }
  if (ranks > 0) w.tab = reinterpret_cast<float*>(take(nh * nqb * ranks * sizeof(float)));
  w.bytes = off;
  return w;
}

static_assert(fwd_smem(2, Bias::bytes(kMaxDistance, kMaxDistance)) <= kHalfSmem && fwd_smem(3, 0) <= kHalfSmem,
              "two forward CTAs share an SM, with the largest table too");
static_assert(dq_smem(2, Bias::bytes(kMaxDistance, kMaxDistance), dq_sums(kMaxBuckets, kMaxDistance), true) <= kMaxSmem &&
                  dkv_smem(3, Bias::bytes(kMaxDistance, kMaxDistance)) <= kMaxSmem,
              "the largest table and its sums fit beside the tiles");

int prepare_attention_window() {
  static std::atomic<unsigned long long> done{0};
  return once_per_device(done, []() -> int {
    const void* all[] = {reinterpret_cast<const void*>(attn_window_fwd_kernel<false>),
                         reinterpret_cast<const void*>(attn_window_fwd_kernel<true>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<0, false>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<1, false>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<1, true>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<2, false>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<2, true>)};
    for (const void* f : all) {
      if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess)
        return set_error(GPIPE_ERR_CUDA, "attention_window: shared-memory attribute failed");
      // a block that is launched with fewer registers than its warps pass on would wait for them for ever
      cudaFuncAttributes at;
      const bool fwd = f == all[0] || f == all[1];
      if (cudaFuncGetAttributes(&at, f) != cudaSuccess || at.numRegs < (fwd ? FWD_REGS : BWD_REGS))
        return set_error(GPIPE_ERR_CUDA, "attention_window: built with fewer registers than its warps share out");
    }
    if (!encode_fn()) return set_error(GPIPE_ERR_CUDA, "attention_window: cuTensorMapEncodeTiled entry point not found");
    return static_cast<int>(GPIPE_OK);
  });
}

// The sizes of one call's tensors.
struct Sizes {
  size_t qkv, o, lse, table, lens;
  Sizes(const WindowArgs& a, int buckets)
      : qkv(static_cast<size_t>(a.nseq) * a.seq * (a.heads + 2 * a.kv_heads) * HD * 2),
        o(static_cast<size_t>(a.nseq) * a.seq * a.heads * HD * 2),
        lse(static_cast<size_t>(a.nseq) * a.seq * a.heads * 4),
        table(static_cast<size_t>(buckets) * a.heads * 4),
        lens(a.lens ? static_cast<size_t>(a.nseq) * 4 : 0) {}
};

int check_launch(const char* what) {
  count_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(GPIPE_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return GPIPE_OK;
}

}  // namespace

int position_bucket_starts(int buckets, int max_distance, int32_t* starts) {
  const int rc = check_buckets(buckets, max_distance);
  if (rc) return rc;
  if (!starts) return set_error(GPIPE_ERR_INVALID_ARG, "position buckets: NULL output");
  bucket_starts(buckets, max_distance, starts);
  return GPIPE_OK;
}

size_t attention_window_scratch_bytes(int nseq, int seq, int heads, int window, int sinks, int buckets) {
  WindowArgs a;
  if (window_args(a, nseq, seq, heads, heads, window, sinks, nullptr, nullptr, 0, 0)) return 0;
  if (buckets != 0 && (buckets < 2 || buckets > kMaxBuckets)) return 0;
  return window_scratch(nullptr, nseq, seq, heads, window, sinks, buckets).bytes;
}

int launch_attention_window_fwd(int nseq, int seq, int heads, int kv_heads, int window, int sinks, const int32_t* lens,
                                const float* table, int buckets, int max_distance, const void* qkv, void* o,
                                float* lse, cudaStream_t s) {
  WindowArgs a;
  int rc = window_args(a, nseq, seq, heads, kv_heads, window, sinks, lens, table, buckets, max_distance);
  if (rc) return rc;
  if (!qkv || !o || !lse || !al16(qkv) || !al16(o))
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_fwd: qkv and o must be 16-B aligned, lse not NULL");
  if (!al4(lse) || !al4(lens) || !al4(table))
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_fwd: lse, lens and table must be aligned to their elements");
  const Sizes size(a, buckets);
  const Range out[] = {{o, size.o}, {lse, size.lse}};
  for (const Range& r : out)
    if (overlaps(r, {{qkv, size.qkv}, {table, size.table}, {lens, size.lens}}) || overlaps(out[0], {out[1]}))
      return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_fwd: o and lse may not overlap each other or the inputs");
  rc = prepare_attention_window();
  if (rc) return rc;
  int* err = device_error_ptr();
  if (!err) return set_error(GPIPE_ERR_CUDA, "attention_window_fwd: no device error word");
  CUtensorMap tq, to;
  if (!make_tmap(&tq, qkv, static_cast<int64_t>(heads + 2 * kv_heads) * HD, seq, nseq, 128) ||
      !make_tmap(&to, o, static_cast<int64_t>(heads) * HD, seq, nseq, 128))
    return set_error(GPIPE_ERR_CUDA, "attention_window_fwd: tensor map creation failed");
  const int grid = ((seq + 127) / 128) * heads * nseq;
  const int smem = a.ranks ? fwd_smem(2, Bias::bytes(a.near[0], a.last)) : fwd_smem(3, 0);
  (void)launch_k<true>(a.ranks ? attn_window_fwd_kernel<true> : attn_window_fwd_kernel<false>, grid, FWD_THREADS,
                       smem, s, tq, to, a, static_cast<__nv_bfloat16*>(o), lse, err);
  return check_launch("attention_window_fwd");
}

int launch_attention_window_bwd(int nseq, int seq, int heads, int kv_heads, int window, int sinks, const int32_t* lens,
                                const float* table, int buckets, int max_distance, const void* qkv, const void* o,
                                const void* dout, const float* lse, void* dqkv, float* dtable_acc, void* scratch,
                                cudaStream_t s) {
  WindowArgs a;
  int rc = window_args(a, nseq, seq, heads, kv_heads, window, sinks, lens, table, buckets, max_distance);
  if (rc) return rc;
  if (!qkv || !o || !dout || !lse || !dqkv || !al16(qkv) || !al16(o) || !al16(dout) || !al16(dqkv))
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "attention_window_bwd: qkv, o, dout and dqkv must be 16-B aligned, lse not NULL");
  if (!al4(lse) || !al4(lens) || !al4(table) || !al4(dtable_acc))
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "attention_window_bwd: lse, lens, table and dtable_acc must be aligned to their elements");
  if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u))
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_bwd: scratch must be 256-B aligned");
  if (dtable_acc && !table)
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_bwd: a table gradient needs the table");
  const WindowScratch w = window_scratch(scratch, nseq, seq, heads, window, sinks, dtable_acc ? a.ranks : 0);
  const Sizes size(a, buckets);
  const Range dx = {dqkv, size.qkv}, tmp = {scratch, w.bytes}, dt = {dtable_acc, dtable_acc ? size.table : 0};
  const Range read[] = {{qkv, size.qkv}, {o, size.o}, {dout, size.o}, {lse, size.lse}, {lens, size.lens}};
  for (const Range& r : read)
    if (overlaps(r, {dx, tmp, dt}))
      return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_bwd: dqkv, dtable_acc and scratch may not overlap the inputs");
  // (the table itself may take its gradient: it is added when nothing reads the table any more)
  if (overlaps(dx, {tmp, dt, {table, size.table}}) || overlaps(tmp, {dt, {table, size.table}}))
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "attention_window_bwd: dqkv, dtable_acc and scratch may not overlap each other or the inputs");
  rc = prepare_attention_window();
  if (rc) return rc;
  int* err = device_error_ptr();
  if (!err) return set_error(GPIPE_ERR_CUDA, "attention_window_bwd: no device error word");
  const int64_t cols = static_cast<int64_t>(heads + 2 * kv_heads) * HD, D = static_cast<int64_t>(heads) * HD;
  CUtensorMap tq64, tq128, td64, td128, tg;
  if (!make_tmap(&tq64, qkv, cols, seq, nseq, 64) || !make_tmap(&tq128, qkv, cols, seq, nseq, 128) ||
      !make_tmap(&td64, dout, D, seq, nseq, 64) || !make_tmap(&td128, dout, D, seq, nseq, 128) ||
      !make_tmap(&tg, dqkv, cols, seq, nseq, 128))
    return set_error(GPIPE_ERR_CUDA, "attention_window_bwd: tensor map creation failed");
  const int64_t prep = static_cast<int64_t>(nseq) * pad128(seq) * heads * 8;
  (void)launch_k(a.ranks ? attn_window_prep_kernel<true> : attn_window_prep_kernel<false>, static_cast<unsigned>((prep + 255) / 256), 256, 0, s, a,
                 static_cast<const __nv_bfloat16*>(qkv), static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, w.ld, w.terms);
  rc = check_launch("attention_window_bwd (prep)");
  if (rc) return rc;
  const int nqb = (seq + 127) / 128, n_dkv = nqb * kv_heads * nseq, n_dq = nqb * heads * nseq;
  // Without wide buckets, what is there for them costs some 2 % (8 x up to 1000 tokens, 12 heads over 4, 32
  // buckets up to 200, forward and backward: 104.5 us instead of 101.8); what they gain is at window_bwd_dq.
  const bool wide = a.near[1] < a.last;
  auto kern = dtable_acc ? (wide ? attn_window_bwd_kernel<2, true> : attn_window_bwd_kernel<2, false>)
              : !a.ranks ? attn_window_bwd_kernel<0, false>
                         : (wide ? attn_window_bwd_kernel<1, true> : attn_window_bwd_kernel<1, false>);
  // Three stages a ring where two CTAs still fit on an SM, or where they do not anyway.  2 x 4096 tokens,
  // 16 heads, everything visible, forward and backward: 391 us with three, 406 us with two (32 buckets up
  // to 128).  With 36 buckets up to 1024 the backward pass takes 370 us with two stages in the dQ CTAs
  // and two CTAs on an SM, 530 us with three and one.
  const int bias_bytes = a.ranks ? Bias::bytes(a.near[1], a.last) : 0;
  const int sums = dtable_acc ? dq_sums(a.ranks, a.last) : 0;
  const bool far = w.far != nullptr;
  auto bytes = [&](int dkv, int dq) {
    const int x = dkv_smem(dkv, bias_bytes), y = dq_smem(dq, bias_bytes, sums, far);
    return x > y ? x : y;
  };
  int dkv_stages = 3, dq_stages = 3;
  if (bytes(2, 2) <= kHalfSmem) {
    if (bytes(3, 2) > kHalfSmem) dkv_stages = 2;
    if (bytes(dkv_stages, 3) > kHalfSmem) dq_stages = 2;
  } else if (bytes(3, 3) > kMaxSmem) {
    dq_stages = 2;
  }
  (void)launch_k(kern, n_dkv + n_dq, BWD_THREADS, bytes(dkv_stages, dq_stages), s, tq64, tq128, td64, td128, tg, a,
                       w, static_cast<const __nv_bfloat16*>(qkv), static_cast<__nv_bfloat16*>(dqkv), n_dkv, dkv_stages,
                       dq_stages, err);
  rc = check_launch("attention_window_bwd");
  if (rc) return rc;
  const int n_sink = w.far ? nseq * kv_heads * a.sinks : 0;
  if (n_sink || dtable_acc) {
    (void)launch_k(attn_window_finish_kernel, n_sink + (dtable_acc ? heads : 0), kFinishThreads, 0, s, a, w,
                   static_cast<__nv_bfloat16*>(dqkv), dtable_acc, n_sink);
    rc = check_launch("attention_window_bwd (finish)");
  }
  return rc;
}

}  // namespace gp
