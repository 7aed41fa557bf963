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
// thread r of the 128 row threads owns row r of every accumulator, and warp 4
// issues every copy and every product.
//
// Scores are kept in the log2 domain: t = s * log2(e) / 8 + bias * log2(e), so
// that an exponential is one ex2.  The bias enters in one of two ways: a tile
// whose distances all lie in the last bucket takes it as a constant; a tile
// nearer to the diagonal reads it from a table by distance in shared memory,
// in which the rows of a warp read consecutive words.
//
// The backward pass uses no atomics, so its results are bit-reproducible:
//   prep    -lse log2(e) and -D of every (head, query), in a layout that the
//           main kernel reads in rows; -inf for padded rows, whose P is then 0.
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
// Every mbarrier wait is bounded as in attention.cu.  The shared-memory tiles'
// layout is described in attention_tiles.cuh.
#include <atomic>
#include <cmath>

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
constexpr float kHidden = -1e30f;  // a table entry at or below it hides its bucket

struct WindowArgs {
  int nseq, seq, heads, kv_heads, window, sinks;
  const int32_t* lens;  // valid tokens per sequence, or NULL: seq
  const float* table;   // [buckets][heads], or NULL
  int ranks;            // non-empty buckets, by rising distance (0: no bias)
  int last;             // first distance of the last of them
  int16_t start[kMaxBuckets];
  uint8_t bucket[kMaxBuckets];
};

__device__ __forceinline__ int seq_len(const WindowArgs& a, int b) {
  return a.lens ? max(0, min(a.lens[b], a.seq)) : a.seq;
}

// A barrier of the 128 row threads on an mbarrier, with the bounded wait: a warp
// that gave up a wait and left its loop cannot strand the others here.
struct RowSync {
  uint64_t* bar;
  int* err;
  volatile int* abort;
  uint32_t phase;
  __device__ __forceinline__ bool operator()() {
    mbar_arrive1(bar);
    return __all_sync(0xffffffffu, await(bar, phase++ & 1u, err, DERR_ACC_WAIT, abort));
  }
};

// The bias by distance, log2 domain: lut[kLutLow + d] for d = -kLutLow ..
// last + kLutHigh - 1 (the last bucket's value from `last` on; a negative
// distance is masked, whatever is read for it).  A tile of 128 x 128 whose
// smallest distance is at most `last` reads no further than last + 254.
constexpr int kLutLow = 128, kLutHigh = 256;
__host__ __device__ constexpr int lut_words(int last) { return (kLutLow + last + kLutHigh + 3) & ~3; }

// Filled by the 128 row threads; val: room for kMaxBuckets floats.
__device__ __forceinline__ bool fill_lut(const WindowArgs& a, int head, float* lut, float* val, int r, RowSync& sync) {
  bool ok = sync();  // nobody reads the previous table any more
  if (r < a.ranks) {
    const float x = a.table[static_cast<int64_t>(a.bucket[r]) * a.heads + head];
    val[r] = x <= kHidden ? -INFINITY : x * kLog2e;
  }
  ok = sync() && ok;
  for (int k = 0; k < a.ranks; ++k) {
    const int from = k == 0 ? -kLutLow : a.start[k];
    const int to = k + 1 < a.ranks ? a.start[k + 1] : a.last + kLutHigh;
    const float x = val[k];
    for (int d = from + r; d < to; d += 128) lut[kLutLow + d] = x;
  }
  return sync() && ok;
}

// Bits 0..x of a word (x < 0: none, x >= 31: all).
__device__ __forceinline__ uint32_t bits_to(int x) {
  return x < 0 ? 0u : (x >= 31 ? 0xffffffffu : (2u << x) - 1u);
}

// Zero rows [from, to) of a tile of 128-byte rows, by one warp, for the async proxy.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to, int lane) {
  for (int x = from * 8 + lane; x < to * 8; x += 32)
    *reinterpret_cast<uint4*>(tile + x * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// Store 64 fp32 TMEM columns of this thread's lane, times scale, as bf16 to dst
// when `valid`; zeros unless `keep` (whatever the accumulator holds then).
__device__ __forceinline__ void store_row64_or_zero(uint32_t taddr, __nv_bfloat16* dst, float scale, bool valid,
                                                    bool keep) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[32];
    ld_row32(taddr + 32 * h, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = keep ? v[i] * scale : 0.f;
    if (valid) {
#pragma unroll
      for (int u = 0; u < 4; ++u) store8(dst + 32 * h + 8 * u, v + 8 * u);
    }
  }
}

__device__ __forceinline__ void zero_row64(__nv_bfloat16* dst) {
#pragma unroll
  for (int u = 0; u < 8; ++u) *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(0u, 0u, 0u, 0u);
}

// The whole warp waits; the answer is the same in every lane.
__device__ __forceinline__ bool warp_await(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* abort) {
  return __all_sync(0xffffffffu, await(bar, parity, err, code, abort));
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
// The hand-offs are those of attention.cu's forward kernel.  Tile t of nt is the
// sinks' narrow block first (where the window has left it), then the window's
// 128-key blocks up to the diagonal.
constexpr int WIN_THREADS = 160;
constexpr int FWD_BAR = 7 * T128;
constexpr int FWD_VAL = FWD_BAR + 128;
constexpr int FWD_LUT = FWD_VAL + kMaxBuckets * 4;

template <bool BIAS>
__global__ void __maxnreg__(168) attn_window_fwd_kernel(const __grid_constant__ CUtensorMap tq,
                                                        const __grid_constant__ WindowArgs a,
                                                        __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                                                        int* err) {
  extern __shared__ __align__(1024) uint8_t sm[];
  if (reinterpret_cast<uintptr_t>(sm) & 1023u) {  // the tiles' swizzle needs 1024-byte alignment
    if (threadIdx.x == 0) atomicExch(err, DERR_ALIGN);
    return;
  }
  uint8_t* sQ = sm;
  uint8_t* sK = sm + T128;      // two buffers
  uint8_t* sV = sm + 3 * T128;  // two buffers
  uint8_t* sP = sm + 5 * T128;  // keys 0..63 | keys 64..127
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + FWD_BAR);
  uint64_t *bq = bar, *bk = bar + 1, *bv = bar + 3, *bs = bar + 5, *bsc = bar + 6, *bp = bar + 7, *bo = bar + 8,
           *bfin = bar + 9, *brow = bar + 10;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 12);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  float* val = reinterpret_cast<float*>(sm + FWD_VAL);
  float* lut = reinterpret_cast<float*>(sm + FWD_LUT);

  const int r = threadIdx.x, warp = r >> 5, ln = r & 31;
  const int nqb = (a.seq + 127) / 128;
  // heads fastest, then sequences, then query blocks from the last (the longest rows first)
  const int h = static_cast<int>(blockIdx.x) % a.heads;
  const int bq_lin = static_cast<int>(blockIdx.x) / a.heads;
  const int b = bq_lin % a.nseq;
  const int qb = nqb - 1 - bq_lin / a.nseq;
  const int q0 = qb * 128, qi = q0 + r;
  const int64_t row0 = static_cast<int64_t>(b) * a.seq;
  const int D = a.heads * HD;
  const int kcol = D + (h / (a.heads / a.kv_heads)) * HD, vcol = kcol + a.kv_heads * HD;

  griddep_wait();
  const int n = seq_len(a, b);
  if (q0 >= n) {  // a block of padding
    if (qi < a.seq && r < 128) {
      zero_row64(out + (row0 + qi) * D + h * HD);
      lse[(row0 + qi) * a.heads + h] = -INFINITY;
    }
    return;
  }
  const int ws = max(0, q0 - a.window + 1) / 128;  // the window's first key block
  const bool sink_tile = a.sinks > 0 && ws > 0;
  const int nt = qb - ws + 1 + (sink_tile ? 1 : 0);
  auto tile_key = [&](int t) { return sink_tile ? (t == 0 ? 0 : (ws + t - 1) * 128) : (ws + t) * 128; };
  auto tile_width = [&](int t) {  // keys of a tile, in steps of 32
    return sink_tile && t == 0 ? (a.sinks + 31) & ~31 : min(128, (n - tile_key(t) + 31) & ~31);
  };

  if (r == 0) {
    prefetch_tmap(&tq);
    for (int i = 0; i < 6; ++i) mbar_init(&bar[i], 1);
    mbar_init(bsc, 128);
    mbar_init(bp, 128);
    mbar_init(bo, 1);
    mbar_init(bfin, 1);
    mbar_init(brow, 128);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tslot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tS = tmem, tO = tmem + 128;

  if (warp == 4) {  // ---- issuer: the warp waits together, lane 0 issues ----
    constexpr uint32_t idO = mma_idesc_bf16(128, 64, false, true);
    int nk[2] = {0, 0}, nv[2] = {0, 0};
    auto load = [&](uint8_t* dst, int col, int row, uint64_t* bar_) {
      if (ln == 0) {
        mbar_arrive_expect_tx(bar_, T128);
        tma_load_3d(dst, &tq, col, row, b, bar_);
      }
    };
    load(sQ, h * HD, q0, bq);
    for (int t = 0; t < 2 && t < nt; ++t) {
      load(sK + t * T128, kcol, tile_key(t), &bk[t]);
      ++nk[t];
      load(sV + t * T128, vcol, tile_key(t), &bv[t]);
      ++nv[t];
    }
    auto issue_s = [&](int t) {  // S_t = Q K_t^T into TMEM (K_t loaded, S_{t-1} read out)
      const uint32_t q = smem_u32(sQ), k = smem_u32(sK + (t & 1) * T128);
      const uint32_t idS = mma_idesc_bf16(128, tile_width(t), false, false);
      if (ln == 0) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tS, kdesc(q, kk), kdesc(k, kk), idS, kk ? 1u : 0u);
        tc_commit(bs);
      }
    };
    bool go = warp_await(bq, 0, err, DERR_MMA_WAIT, abort) && warp_await(&bk[0], 0, err, DERR_MMA_WAIT, abort);
    if (go) {
      tc_fence_after();
      issue_s(0);
    }
    for (int t = 0; t < nt && go; ++t) {
      const int kb = t & 1;
      if (t + 1 < nt) {  // S_{t+1} as soon as the rows have read S_t: it computes during tile t's softmax
        if (!warp_await(&bk[(t + 1) & 1], ((t + 1) >> 1) & 1, err, DERR_MMA_WAIT, abort)) break;
        if (!warp_await(bsc, t & 1, err, DERR_MMA_WAIT, abort)) break;
        tc_fence_after();
        issue_s(t + 1);
        if (t + 2 < nt) {  // K buffer of tile t: S_t is done
          load(sK + kb * T128, kcol, tile_key(t + 2), &bk[kb]);
          ++nk[kb];
        }
      }
      if (!warp_await(&bv[kb], (t >> 1) & 1, err, DERR_MMA_WAIT, abort)) break;
      const int w = tile_width(t), left = n - tile_key(t);
      if (left < w) {  // values behind the sequence's end: their P is 0, they themselves may be anything
        zero_rows(sV + kb * T128, left, w, ln);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!warp_await(bp, t & 1, err, DERR_MMA_WAIT, abort)) break;                 // P_t written, O rescaled
      if (t > 0 && !warp_await(bo, (t - 1) & 1, err, DERR_MMA_WAIT, abort)) break;  // O += P_{t-1} V_{t-1} done
      if (t >= 1 && t + 1 < nt) {                                                  // V buffer of tile t-1 is free
        const int nb = (t + 1) & 1;
        load(sV + nb * T128, vcol, tile_key(t + 1), &bv[nb]);
        ++nv[nb];
      }
      tc_fence_after();
      if (ln == 0) {
        const uint32_t p = smem_u32(sP), v = smem_u32(sV + kb * T128);
        for (int kk = 0; kk < w / 16; ++kk)
          tc_mma_f16(tO, kdesc(p + (kk >> 2) * T128, kk & 3), mndesc(v, kk), idO, (t | kk) ? 1u : 0u);
        tc_commit(bo);
      }
    }
    // no copy may still be landing, and no product still running, when the CTA exits
    if (ln == 0) {
      tc_commit(bfin);
      mbar_wait_bounded(bfin, 0, err, DERR_DRAIN_WAIT);
      for (int bb = 0; bb < 2; ++bb) {
        if (nk[bb]) mbar_wait_bounded(&bk[bb], (nk[bb] - 1) & 1, err, DERR_DRAIN_WAIT);
        if (nv[bb]) mbar_wait_bounded(&bv[bb], (nv[bb] - 1) & 1, err, DERR_DRAIN_WAIT);
      }
      mbar_wait_bounded(bq, 0, err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else {  // ---- rows ----
    const uint32_t lane = static_cast<uint32_t>(warp * 32) << 16;
    RowSync sync{brow, err, abort, 0u};
    float m = -INFINITY, l = 0.f;
    bool ok = !BIAS || fill_lut(a, h, lut, val, r, sync);
    for (int t = 0; t < nt && ok; ++t) {
      const int j0 = tile_key(t), w = tile_width(t);
      ok = warp_await(bs, t & 1, err, DERR_ACC_WAIT, abort);
      if (!ok) break;
      tc_fence_after();
      float sv[128];
      {
        // columns behind the tile's width hold what was there before: the mask hides them
        const uint32_t at[4] = {tS + lane, tS + lane + 32, tS + lane + 64, tS + lane + 96};
        ld_rows<4>(at, sv);
      }
      tc_fence_before();
      mbar_arrive1(bsc);  // S may be overwritten by the next tile's product
      // scores = sc * s + cb (log2 domain): the raw scores with a constant bias,
      // or with the bias by distance already added
      float sc = kScaleLog2, cb = 0.f;
      if (BIAS) {
        if (q0 - (j0 + 127) >= a.last) {
          cb = lut[kLutLow + a.last];
        } else {
          const float* at = lut + kLutLow + (qi - j0);
#pragma unroll
          for (int i = 0; i < 128; ++i) sv[i] = fmaf(sv[i], kScaleLog2, at[-i]);
          sc = 1.f;
        }
      }
      if (w < 128 || !(j0 + 127 <= q0 && q0 + 127 - j0 < a.window)) {  // some pair is hidden
        const int hi = qi - j0, lo = hi - a.window + 1, sk = a.sinks - j0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t see = bits_to(hi - 32 * c) & (~bits_to(lo - 1 - 32 * c) | bits_to(sk - 1 - 32 * c));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((see >> i) & 1u)) sv[32 * c + i] = -INFINITY;
        }
      }
      float mx8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
#pragma unroll
      for (int i = 0; i < 128; i += 2) mx8[(i >> 1) & 7] = fmax3(mx8[(i >> 1) & 7], sv[i], sv[i + 1]);
      const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
      const float mn = fmaxf(m, fmaf(mx, sc, cb));
      const float ms = mn == -INFINITY ? 0.f : mn;  // nothing visible yet: exp2(-inf - 0) = 0
      const float alpha = ex2_approx(m - ms);
      m = mn;
      if (t > 0) {  // the previous O product reads P and writes O
        ok = warp_await(bo, (t - 1) & 1, err, DERR_ACC_WAIT, abort);
        if (!ok) break;
        tc_fence_after();
      }
      const float off = cb - ms;
      float rs8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (32 * c < w) {
          float* pc = sv + 32 * c;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            ffma2(pc[i], pc[i + 1], pc[i], pc[i + 1], sc, sc, off, off);
            pc[i] = ex2_approx(pc[i]);
            pc[i + 1] = ex2_approx(pc[i + 1]);
            const int e = (i >> 1) & 3;
            fadd2(rs8[2 * e], rs8[2 * e + 1], rs8[2 * e], rs8[2 * e + 1], pc[i], pc[i + 1]);
          }
          st_row32_bf16(sP + (c >> 1) * T128, r, (c & 1) * 4, pc);
        }
      }
      const float rs = ((rs8[0] + rs8[1]) + (rs8[2] + rs8[3])) + ((rs8[4] + rs8[5]) + (rs8[6] + rs8[7]));
      if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {  // warp-uniform: tcgen05 loads/stores are per warp
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t u[32];
          tmem_ld32(tO + lane + 32 * c, u);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a0, a1;
            fmul2(a0, a1, __uint_as_float(u[i]), __uint_as_float(u[i + 1]), alpha, alpha);
            u[i] = __float_as_uint(a0);
            u[i + 1] = __float_as_uint(a1);
          }
          tmem_st32(tO + lane + 32 * c, u);
        }
        tmem_st_wait();
      }
      l = l * alpha + rs;
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive1(bp);
    }
    if (ok) ok = warp_await(bo, (nt - 1) & 1, err, DERR_ACC_WAIT, abort);
    tc_fence_after();
    if (ok) {
      // l = 0: a row that sees nothing (padding, or every bucket of its keys hidden)
      store_row64_or_zero(tO + lane, out + (row0 + qi) * D + h * HD, 1.0f / l, qi < a.seq, qi < n && l != 0.f);
      if (qi < a.seq) lse[(row0 + qi) * a.heads + h] = qi < n && l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
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
//   far    float [nseq][heads][query blocks][sinks][128]: dV | dK of the sinks from one query block
//   base   float [nseq][kv_heads][sinks][128]: their dV | dK from the queries near them
//   tab    float [nseq][query blocks][heads][ranks]: dtable from one query block
struct WindowScratch {
  float2* ld;
  float* far;   // NULL: no query block is far from the sinks
  float* base;
  float* tab;   // NULL: no table gradient
  size_t bytes;
};

__host__ __device__ constexpr int pad128(int x) { return (x + 127) / 128 * 128; }
// The first query block whose window has left the first key block.
__host__ __device__ constexpr int first_far_block(int window) { return (window + 254) / 128; }

__global__ void __launch_bounds__(256) attn_window_prep_kernel(const __grid_constant__ WindowArgs a,
                                                               const __nv_bfloat16* __restrict__ o,
                                                               const __nv_bfloat16* __restrict__ dout,
                                                               const float* __restrict__ lse, float2* __restrict__ ld) {
  griddep_wait();
  griddep_launch();
  // eight threads per (sequence, query, head), each 8 of the 64 columns
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const int sub = threadIdx.x & 7;
  const int seqpad = pad128(a.seq);
  const int h = static_cast<int>(item % a.heads);
  const int64_t bi = item / a.heads;
  const int i = static_cast<int>(bi % seqpad);
  const int64_t b = bi / seqpad;
  const bool in = b < a.nseq;
  const bool live = in && i < seq_len(a, static_cast<int>(in ? b : 0));
  float d = 0.f, L = -INFINITY;
  if (live) {
    const int64_t row = (b * a.seq + i) * a.heads + h;
    float x[8], y[8];
    load8(o + row * HD + 8 * sub, x);
    load8(dout + row * HD + 8 * sub, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) d = fmaf(x[e], y[e], d);
    const float v = lse[row];
    L = v == -INFINITY ? -INFINITY : -v * kLog2e;  // a row that sees nothing: P = 0
  }
#pragma unroll
  for (int s = 4; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
  if (in && sub == 0) ld[(b * a.heads + h) * seqpad + i] = make_float2(L, -d);
}

constexpr int BWD_TILES = 6 * T128;
constexpr int BWD_LD = BWD_TILES;  // dK/dV: -LSE and -D of two query blocks (1 KB)
constexpr int BWD_BAR = BWD_LD + 4 * 64 * 4;
constexpr int BWD_VAL = BWD_BAR + 128;
constexpr int BWD_LUT = BWD_VAL + kMaxBuckets * 4;

// MODE 0: no bias; 1: bias; 2: bias and its gradient.
//
// dQ CTA.  Key blocks of 64 by rising key, the sinks' block last.  In the
// gradient of the table a row's distances fall along the walk, so its bucket
// falls too: the running sums of dS and P are added to the row's own word of
// the bucket (no two threads share one) where a bucket ends.
template <int MODE>
__device__ void window_bwd_dq(const WindowArgs& a, const CUtensorMap* tq64, const CUtensorMap* tq128,
                              const CUtensorMap* td128, const WindowScratch& ws_, __nv_bfloat16* __restrict__ dqkv,
                              int item, int* err, uint8_t* sm) {
  uint8_t* sQ = sm;
  uint8_t* sdO = sm + T128;
  uint8_t* sKV = sm + 2 * T128;  // two slots of K (64 rows) | V (64 rows)
  uint8_t* sP = sm + 4 * T128;   // 128 queries x 64 keys (the sinks' block only)
  uint8_t* sdS = sm + 5 * T128;  // 128 queries x 64 keys
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + BWD_BAR);
  uint64_t *bq = bar, *bkv = bar + 1, *bs = bar + 3, *bsc = bar + 4, *bp = bar + 5, *bo = bar + 6, *bfin = bar + 7,
           *brow = bar + 10;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 12);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  float* val = reinterpret_cast<float*>(sm + BWD_VAL);
  float* lut = reinterpret_cast<float*>(sm + BWD_LUT);
  float* accS = lut + lut_words(a.last);   // [ranks][128]
  float* accP = accS + a.ranks * 128;      // [ranks][128]
  uint32_t* ends = reinterpret_cast<uint32_t*>(accP + a.ranks * 128);  // bit d: distance d is its bucket's first

  const int r = threadIdx.x, warp = r >> 5, ln = r & 31;
  const int nqb = (a.seq + 127) / 128;
  const int h = item % a.heads;
  const int b = (item / a.heads) % a.nseq;
  const int qb = nqb - 1 - item / (a.heads * a.nseq);
  const int q0 = qb * 128, qi = q0 + r;
  const int64_t row0 = static_cast<int64_t>(b) * a.seq;
  const int D = a.heads * HD;
  const int64_t ld = static_cast<int64_t>(a.heads + 2 * a.kv_heads) * HD;
  const int kcol = D + (h / (a.heads / a.kv_heads)) * HD, vcol = kcol + a.kv_heads * HD;

  griddep_wait();
  const int n = seq_len(a, b);
  float* tab = MODE == 2 ? ws_.tab + ((static_cast<int64_t>(b) * nqb + qb) * a.heads + h) * a.ranks : nullptr;
  if (q0 >= n) {  // a block of padding
    if (qi < a.seq && r < 128) zero_row64(dqkv + (row0 + qi) * ld + h * HD);
    if (MODE == 2 && r < a.ranks) tab[r] = 0.f;
    return;
  }
  const bool sink_tile = a.sinks > 0 && qb >= first_far_block(a.window);
  const int kb0 = a.sinks > 0 && !sink_tile ? 0 : max(0, q0 - a.window + 1) / 64;
  const int nwin = min(q0 + 127, n - 1) / 64 - kb0 + 1;
  const int nt = nwin + (sink_tile ? 1 : 0);
  auto tile_key = [&](int t) { return t < nwin ? (kb0 + t) * 64 : 0; };

  if (r == 0) {
    prefetch_tmap(tq64);
    prefetch_tmap(tq128);
    prefetch_tmap(td128);
    for (int i = 0; i < 4; ++i) mbar_init(&bar[i], 1);
    mbar_init(bsc, 128);
    mbar_init(bp, 128);
    mbar_init(bo, 1);
    mbar_init(bfin, 1);
    mbar_init(brow, 128);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tslot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tS = tmem, tP = tmem + 64, tQ = tmem + 128;

  if (warp == 4) {  // ---- issuer ----
    constexpr uint32_t idSP = mma_idesc_bf16(128, 64, false, false);
    constexpr uint32_t idQ = mma_idesc_bf16(128, 64, false, true);
    constexpr uint32_t idT = mma_idesc_bf16(128, 64, true, true);
    int nkv[2] = {0, 0};
    if (ln == 0) {
      mbar_arrive_expect_tx(bq, 2 * T128);
      tma_load_3d(sQ, tq128, h * HD, q0, b, bq);
      tma_load_3d(sdO, td128, h * HD, q0, b, bq);
    }
    auto load_kv = [&](int t) {
      const int s = t & 1;
      if (ln == 0) {
        mbar_arrive_expect_tx(&bkv[s], 2 * T64);
        tma_load_3d(sKV + s * T128, tq64, kcol, tile_key(t), b, &bkv[s]);
        tma_load_3d(sKV + s * T128 + T64, tq64, vcol, tile_key(t), b, &bkv[s]);
      }
      ++nkv[s];
    };
    for (int t = 0; t < 2 && t < nt; ++t) load_kv(t);
    auto issue_sp = [&](int t) {  // S = Q K_t^T, dP = dO V_t^T (tile t loaded, tile t-1's read out)
      uint8_t* kv = sKV + (t & 1) * T128;
      const int left = n - tile_key(t);
      if (left < 64) {  // keys behind the sequence's end: P = dS = 0, the rows themselves may be anything
        zero_rows(kv, left, 64, ln);
        zero_rows(kv + T64, left, 64, ln);
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t q = smem_u32(sQ), dO = smem_u32(sdO), k = smem_u32(kv), v = smem_u32(kv + T64);
      if (ln == 0) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tS, kdesc(q, kk), kdesc(k, kk), idSP, kk ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tP, kdesc(dO, kk), kdesc(v, kk), idSP, kk ? 1u : 0u);
        tc_commit(bs);
      }
    };
    bool go = warp_await(bq, 0, err, DERR_MMA_WAIT, abort) && warp_await(&bkv[0], 0, err, DERR_MMA_WAIT, abort);
    if (go) {
      if (n - q0 < 128) {  // padded queries: with Q = dO = 0 and P = 0 they add nothing to the sinks' sums
        zero_rows(sQ, n - q0, 128, ln);
        zero_rows(sdO, n - q0, 128, ln);
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      issue_sp(0);
    }
    for (int t = 0; t < nt && go; ++t) {
      if (t + 1 < nt) {  // the next tile's S, dP as soon as the rows have read tile t's
        if (!warp_await(&bkv[(t + 1) & 1], ((t + 1) >> 1) & 1, err, DERR_MMA_WAIT, abort)) break;
        if (!warp_await(bsc, t & 1, err, DERR_MMA_WAIT, abort)) break;
        tc_fence_after();
        issue_sp(t + 1);
      }
      if (!warp_await(bp, t & 1, err, DERR_MMA_WAIT, abort)) break;  // dS_t written
      tc_fence_after();
      if (ln == 0) {
        const uint32_t ds = smem_u32(sdS), k = smem_u32(sKV + (t & 1) * T128);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tQ, kdesc(ds, kk), mndesc(k, kk), idQ, (t | kk) ? 1u : 0u);
        if (t >= nwin) {
          // the sinks' dV = P^T dO and dK = dS^T Q over this block's queries, in the columns of S and
          // dP: P and dS read MN-major.  Rows 64..127 of the products come from the addresses 1024
          // bytes further (inside the CTA's shared memory) and are not read.
          const uint32_t p = smem_u32(sP), q = smem_u32(sQ), dO = smem_u32(sdO);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_f16(tS, sw128_desc(p + kk * 2048, 1024, 1024), mndesc(dO, kk), idT, kk ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_f16(tP, sw128_desc(ds + kk * 2048, 1024, 1024), mndesc(q, kk), idT, kk ? 1u : 0u);
        }
        tc_commit(bo);
      }
      if (t + 2 < nt) {  // tile t's slot, once dQ += dS_t K_t is done
        if (!warp_await(bo, t & 1, err, DERR_MMA_WAIT, abort)) break;
        load_kv(t + 2);
      }
    }
    if (ln == 0) {
      tc_commit(bfin);
      mbar_wait_bounded(bfin, 0, err, DERR_DRAIN_WAIT);
      for (int s = 0; s < 2; ++s)
        if (nkv[s]) mbar_wait_bounded(&bkv[s], (nkv[s] - 1) & 1, err, DERR_DRAIN_WAIT);
      mbar_wait_bounded(bq, 0, err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else {  // ---- rows ----
    const uint32_t lane = static_cast<uint32_t>(warp * 32) << 16;
    RowSync sync{brow, err, abort, 0u};
    bool ok = !MODE || fill_lut(a, h, lut, val, r, sync);
    int rank = -1;                   // the bucket (by rank) of the running sums
    float runS = 0.f, runP = 0.f;
    const int nend = a.last / 32 + 1;
    if (MODE == 2) {
      for (int k = 0; k < 2 * a.ranks; ++k) accS[k * 128 + r] = 0.f;
      for (int x = r; x < nend; x += 128) ends[x] = 0u;
      ok = sync() && ok;
      if (r < a.ranks) atomicOr(&ends[a.start[r] >> 5], 1u << (a.start[r] & 31));
      ok = sync() && ok;
    }
    auto rank_of = [&](int d) {
      int k = a.ranks - 1;
      while (k > 0 && a.start[k] > d) --k;
      return k;
    };
    auto flush = [&]() {
      if (rank >= 0) {
        accS[rank * 128 + r] += runS;
        accP[rank * 128 + r] += runP;
      }
      runS = runP = 0.f;
    };
    if (MODE == 2) rank = rank_of(qi - kb0 * 64);
    const float2 LD = ws_.ld[(static_cast<int64_t>(b) * a.heads + h) * pad128(a.seq) + qi];
    for (int t = 0; t < nt && ok; ++t) {
      const int j0 = tile_key(t);
      const bool sink = t >= nwin;
      ok = warp_await(bs, t & 1, err, DERR_ACC_WAIT, abort);
      if (!ok) break;
      tc_fence_after();
      float v[128];  // S (64 columns), then dP (64 columns), one round trip
      {
        const uint32_t at[4] = {tS + lane, tS + lane + 32, tP + lane, tP + lane + 32};
        ld_rows<4>(at, v);
      }
      tc_fence_before();
      mbar_arrive1(bsc);
      const bool near = MODE && q0 - (j0 + 63) <= a.last;  // not all pairs inside the last bucket
      if (near) {
        const float* bias = lut + kLutLow + (qi - j0);
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = fmaf(v[i], kScaleLog2, bias[-i] + LD.x);
      } else {
        const float c = (MODE ? lut[kLutLow + a.last] : 0.f) + LD.x;
#pragma unroll
        for (int i = 0; i < 64; i += 2) ffma2(v[i], v[i + 1], v[i], v[i + 1], kScaleLog2, kScaleLog2, c, c);
      }
      if (sink || !(j0 + 63 <= q0 && (q0 + 127 - j0 < a.window || j0 + 64 <= a.sinks))) {
        const int hi = qi - j0, lo = hi - a.window + 1, sk = a.sinks - j0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t near_bits = sink ? 0u : ~bits_to(lo - 1 - 32 * c);
          const uint32_t see = bits_to(hi - 32 * c) & (near_bits | bits_to(sk - 1 - 32 * c));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((see >> i) & 1u)) v[32 * c + i] = -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        v[i] = ex2_approx(v[i]);  // P
        v[i + 1] = ex2_approx(v[i + 1]);
        float d0, d1;
        fadd2(d0, d1, v[64 + i], v[65 + i], LD.y, LD.y);
        fmul2(v[64 + i], v[65 + i], v[i], v[i + 1], d0, d1);  // dS
      }
      if (MODE == 2) {
        if (sink) {  // distances start again, further away
          flush();
          rank = rank_of(qi);
        }
        if (near) {
          // bit i: column i ends its bucket (distance qi - j0 - i is the bucket's first)
          uint64_t stop = 0;
          const int top = qi - j0;  // distance of column 0
#pragma unroll
          for (int i = 0; i < 64; i += 32) {
            // distances top - i - 31 .. top - i, lowest first, from the bitmap; reversed
            const int d = top - i - 31;
            const int q = d >> 5, s = d & 31;  // floor division
            const uint32_t w0 = q >= 0 && q < nend ? ends[q] : 0u;
            const uint32_t w1 = q + 1 >= 0 && q + 1 < nend ? ends[q + 1] : 0u;
            stop |= static_cast<uint64_t>(__brev(__funnelshift_r(w0, w1, s))) << i;
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            runS += v[64 + i];
            runP += v[i];
            if ((stop >> i) & 1u) {
              flush();
              --rank;
            }
          }
        } else {
          float s4[4] = {0.f, 0.f, 0.f, 0.f}, p4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            fadd2(s4[0], s4[1], s4[0], s4[1], v[64 + i], v[65 + i]);
            fadd2(s4[2], s4[3], s4[2], s4[3], v[66 + i], v[67 + i]);
            fadd2(p4[0], p4[1], p4[0], p4[1], v[i], v[i + 1]);
            fadd2(p4[2], p4[3], p4[2], p4[3], v[i + 2], v[i + 3]);
          }
          runS += (s4[0] + s4[1]) + (s4[2] + s4[3]);
          runP += (p4[0] + p4[1]) + (p4[2] + p4[3]);
        }
      }
      if (t > 0) {  // the previous dQ product reads the dS tile
        ok = warp_await(bo, (t - 1) & 1, err, DERR_ACC_WAIT, abort);
        if (!ok) break;
      }
      if (sink) {
        st_row32_bf16(sP, r, 0, v);
        st_row32_bf16(sP, r, 4, v + 32);
      }
      st_row32_bf16(sdS, r, 0, v + 64);
      st_row32_bf16(sdS, r, 4, v + 96);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive1(bp);
    }
    if (ok) ok = warp_await(bo, (nt - 1) & 1, err, DERR_ACC_WAIT, abort);
    tc_fence_after();
    if (ok) {
      store_row64_or_zero(tQ + lane, dqkv + (row0 + qi) * ld + h * HD, 0.125f, qi < a.seq, qi < n);
      if (sink_tile) {
        float* part = ws_.far + (((static_cast<int64_t>(b) * a.heads + h) * nqb + qb) * a.sinks + r) * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // dV | dK
          float x[32];
          ld_row32((c < 2 ? tS : tP) + lane + 32 * (c & 1), x);
          if (r < a.sinks) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) store8(part + 32 * c + i, x + i);
          }
        }
      }
    }
    if (MODE == 2) {
      flush();
      float e = 0.f;  // the error of D: the row's dS sum to it instead of 0
      for (int k = 0; k < a.ranks; ++k) e += accS[k * 128 + r];
      for (int k = 0; k < a.ranks; ++k) {
        const float x = accS[k * 128 + r] - e * accP[k * 128 + r];
        accS[k * 128 + r] = qi < n ? x : 0.f;
      }
      sync();
      for (int k = warp; k < a.ranks; k += 4) {
        const float* row = accS + k * 128;
        const float x = warp_sum((row[ln] + row[ln + 32]) + (row[ln + 64] + row[ln + 96]));
        if (ln == 0) tab[k] = x;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// dK/dV CTA of 128 keys of one key/value head: iterations t = 0 .. group * nq - 1
// over the 64-query blocks that see them, one query head after the other.
template <int MODE>
__device__ void window_bwd_dkv(const WindowArgs& a, const CUtensorMap* tq64, const CUtensorMap* tq128,
                               const CUtensorMap* td64, const WindowScratch& ws_, __nv_bfloat16* __restrict__ dqkv,
                               int item, int* err, uint8_t* sm) {
  uint8_t* sK = sm;
  uint8_t* sV = sm + T128;
  uint8_t* sQ = sm + 2 * T128;   // two slots of Q (64 rows) | dO (64 rows)
  uint8_t* sPt = sm + 4 * T128;  // 128 keys x 64 queries
  uint8_t* sdSt = sm + 5 * T128; // 128 keys x 64 queries
  float* sL = reinterpret_cast<float*>(sm + BWD_LD);  // [2][64] -LSE (log2 domain)
  float* sD = sL + 128;                               // [2][64] -D
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + BWD_BAR);
  uint64_t *bkv = bar, *bq = bar + 1, *bs = bar + 3, *bsc = bar + 4, *bp = bar + 5, *bo = bar + 6, *bfin = bar + 7,
           *bld = bar + 8,  // bld[2]: the LSE and D of a block are in their slot (64 writers)
           *brow = bar + 10;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 12);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  float* val = reinterpret_cast<float*>(sm + BWD_VAL);
  float* lut = reinterpret_cast<float*>(sm + BWD_LUT);

  const int r = threadIdx.x, warp = r >> 5, ln = r & 31;
  const int kvh = item % a.kv_heads;
  const int b = (item / a.kv_heads) % a.nseq;
  const int kb = item / (a.kv_heads * a.nseq);  // by rising key: in a full causal pass the longest first
  const int group = a.heads / a.kv_heads, h0 = kvh * group;
  const int k0 = kb * 128, kr = k0 + r;
  const int64_t row0 = static_cast<int64_t>(b) * a.seq;
  const int D = a.heads * HD;
  const int64_t ld = static_cast<int64_t>(a.heads + 2 * a.kv_heads) * HD;
  const int kcol = D + kvh * HD, vcol = kcol + a.kv_heads * HD;
  const int seqpad = pad128(a.seq);

  griddep_wait();
  const int n = seq_len(a, b);
  if (k0 >= n) {  // a block of padding
    if (kr < a.seq && r < 128) {
      zero_row64(dqkv + (row0 + kr) * ld + kcol);
      zero_row64(dqkv + (row0 + kr) * ld + vcol);
    }
    return;
  }
  // the queries of this block: those whose window reaches it, and, for the sinks' block, the rest of
  // the 128-query blocks whose window reaches it (the dQ CTAs of the others account for the sinks)
  const int i0 = k0 / 64;
  const int imax = min(n - 1, kb == 0 && a.sinks > 0 ? first_far_block(a.window) * 128 - 1 : k0 + 127 + a.window - 1);
  const int nq = imax / 64 - i0 + 1;
  const int niter = group * nq;

  if (r == 0) {
    prefetch_tmap(tq64);
    prefetch_tmap(tq128);
    prefetch_tmap(td64);
    for (int i = 0; i < 4; ++i) mbar_init(&bar[i], 1);
    mbar_init(bsc, 128);
    mbar_init(bp, 128);
    mbar_init(bo, 1);
    mbar_init(bfin, 1);
    mbar_init(&bld[0], 64);
    mbar_init(&bld[1], 64);
    mbar_init(brow, 128);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tslot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tS = tmem, tP = tmem + 64, tV = tmem + 128, tK = tmem + 192;

  if (warp == 4) {  // ---- issuer ----
    constexpr uint32_t idSP = mma_idesc_bf16(128, 64, false, false);
    constexpr uint32_t idKV = mma_idesc_bf16(128, 64, false, true);
    int nqi[2] = {0, 0};
    if (ln == 0) {
      mbar_arrive_expect_tx(bkv, 2 * T128);
      tma_load_3d(sK, tq128, kcol, k0, b, bkv);
      tma_load_3d(sV, tq128, vcol, k0, b, bkv);
    }
    auto load_q = [&](int t) {
      const int s = t & 1;
      if (ln == 0) {
        const int h = h0 + t / nq, q0 = (i0 + t % nq) * 64;
        mbar_arrive_expect_tx(&bq[s], 2 * T64);
        tma_load_3d(sQ + s * T128, tq64, h * HD, q0, b, &bq[s]);
        tma_load_3d(sQ + s * T128 + T64, td64, h * HD, q0, b, &bq[s]);
      }
      ++nqi[s];
    };
    for (int t = 0; t < 2 && t < niter; ++t) load_q(t);
    auto issue_sp = [&](int t) {  // S^T = K Q_t^T, dP^T = V dO_t^T
      uint8_t* qd = sQ + (t & 1) * T128;
      const int left = n - (i0 + t % nq) * 64;
      if (left < 64) {  // padded queries: P = dS = 0, the rows themselves may be anything
        zero_rows(qd, left, 64, ln);
        zero_rows(qd + T64, left, 64, ln);
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t k = smem_u32(sK), v = smem_u32(sV), q = smem_u32(qd), dO = smem_u32(qd + T64);
      if (ln == 0) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tS, kdesc(k, kk), kdesc(q, kk), idSP, kk ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tP, kdesc(v, kk), kdesc(dO, kk), idSP, kk ? 1u : 0u);
        tc_commit(bs);
      }
    };
    bool go = warp_await(bkv, 0, err, DERR_MMA_WAIT, abort) && warp_await(&bq[0], 0, err, DERR_MMA_WAIT, abort);
    if (go) {
      tc_fence_after();
      issue_sp(0);
    }
    for (int t = 0; t < niter && go; ++t) {
      if (t + 1 < niter) {  // the next block's S^T, dP^T as soon as the rows have read block t's
        if (!warp_await(&bq[(t + 1) & 1], ((t + 1) >> 1) & 1, err, DERR_MMA_WAIT, abort)) break;
        if (!warp_await(bsc, t & 1, err, DERR_MMA_WAIT, abort)) break;
        tc_fence_after();
        issue_sp(t + 1);
      }
      if (!warp_await(bp, t & 1, err, DERR_MMA_WAIT, abort)) break;  // P^T, dS^T of block t written
      tc_fence_after();
      if (ln == 0) {
        const uint32_t pt = smem_u32(sPt), dst = smem_u32(sdSt), q = smem_u32(sQ + (t & 1) * T128), dO = q + T64;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tV, kdesc(pt, kk), mndesc(dO, kk), idKV, (t | kk) ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tK, kdesc(dst, kk), mndesc(q, kk), idKV, (t | kk) ? 1u : 0u);
        tc_commit(bo);
      }
      if (t + 2 < niter) {  // block t's slot, once dV, dK of block t are done
        if (!warp_await(bo, t & 1, err, DERR_MMA_WAIT, abort)) break;
        load_q(t + 2);
      }
    }
    if (ln == 0) {
      tc_commit(bfin);
      mbar_wait_bounded(bfin, 0, err, DERR_DRAIN_WAIT);
      for (int s = 0; s < 2; ++s)
        if (nqi[s]) mbar_wait_bounded(&bq[s], (nqi[s] - 1) & 1, err, DERR_DRAIN_WAIT);
      mbar_wait_bounded(bkv, 0, err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else {  // ---- rows ----
    const uint32_t lane = static_cast<uint32_t>(warp * 32) << 16;
    // -LSE and -D of a block's 64 queries, each read one block ahead; block t sits in slot t & 1 and is
    // published by the (t >> 1)-th phase of bld[t & 1]
    auto ld_at = [&](int t) {
      return ws_.ld[(static_cast<int64_t>(b) * a.heads + h0 + t / nq) * seqpad + (i0 + t % nq) * 64 + r];
    };
    if (r < 64) {
      const float2 x = ld_at(0);
      sL[r] = x.x;
      sD[r] = x.y;
      mbar_arrive1(&bld[0]);
    }
    RowSync sync{brow, err, abort, 0u};
    bool ok = true;
    for (int t = 0; t < niter; ++t) {
      const int q0 = (i0 + t % nq) * 64, s = t & 1;
      if (MODE && t % nq == 0) ok = fill_lut(a, h0 + t / nq, lut, val, r, sync);
      if (ok) ok = warp_await(&bld[s], (t >> 1) & 1, err, DERR_ACC_WAIT, abort);
      float2 next = make_float2(0.f, 0.f);
      if (r < 64 && t + 1 < niter) next = ld_at(t + 1);
      if (ok) ok = warp_await(bs, t & 1, err, DERR_ACC_WAIT, abort);
      if (!ok) break;
      tc_fence_after();
      float v[128];  // S^T (64 columns), then dP^T (64 columns), one round trip
      {
        const uint32_t at[4] = {tS + lane, tS + lane + 32, tP + lane, tP + lane + 32};
        ld_rows<4>(at, v);
      }
      tc_fence_before();
      mbar_arrive1(bsc);
      const float* L = sL + s * 64;
      const float* Dq = sD + s * 64;
      if (MODE && q0 - (k0 + 127) < a.last) {
        const float* bias = lut + kLutLow + (q0 - kr);
#pragma unroll
        for (int q = 0; q < 64; ++q) v[q] = fmaf(v[q], kScaleLog2, bias[q] + L[q]);
      } else {
        const float c = MODE ? lut[kLutLow + a.last] : 0.f;
#pragma unroll
        for (int q = 0; q < 64; q += 2) {
          float l0 = L[q], l1 = L[q + 1];
          if (MODE) fadd2(l0, l1, l0, l1, c, c);
          ffma2(v[q], v[q + 1], v[q], v[q + 1], kScaleLog2, kScaleLog2, l0, l1);
        }
      }
      if (!(q0 >= k0 + 127 && q0 + 63 - k0 < a.window)) {  // some pair may be hidden
        const int lo = kr - q0, hi = kr < a.sinks ? 63 : lo + a.window - 1;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t see = bits_to(hi - 32 * c) & ~bits_to(lo - 1 - 32 * c);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((see >> i) & 1u)) v[32 * c + i] = -INFINITY;
        }
      }
#pragma unroll
      for (int q = 0; q < 64; q += 2) {
        v[q] = ex2_approx(v[q]);  // P^T
        v[q + 1] = ex2_approx(v[q + 1]);
        float d0, d1;
        fadd2(d0, d1, v[64 + q], v[65 + q], Dq[q], Dq[q + 1]);
        fmul2(v[64 + q], v[65 + q], v[q], v[q + 1], d0, d1);  // dS^T
      }
      if (t > 0) {  // the previous dV, dK products read the P^T and dS^T tiles
        ok = warp_await(bo, (t - 1) & 1, err, DERR_ACC_WAIT, abort);
        if (!ok) break;
      }
      st_row32_bf16(sPt, r, 0, v);
      st_row32_bf16(sPt, r, 4, v + 32);
      st_row32_bf16(sdSt, r, 0, v + 64);
      st_row32_bf16(sdSt, r, 4, v + 96);
      if (r < 64 && t + 1 < niter) {  // the next block's
        sL[(s ^ 1) * 64 + r] = next.x;
        sD[(s ^ 1) * 64 + r] = next.y;
        mbar_arrive1(&bld[s ^ 1]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive1(bp);
    }
    if (ok) ok = warp_await(bo, (niter - 1) & 1, err, DERR_ACC_WAIT, abort);
    tc_fence_after();
    if (ok) {
      // the sinks' rows go on to the finish kernel, where query blocks far from them add to them
      const bool on = ws_.far && kr < a.sinks && kr < n;
      __nv_bfloat16* dst = dqkv + (row0 + kr) * ld;
      store_row64_or_zero(tK + lane, dst + kcol, 0.125f, kr < a.seq && !on, kr < n);
      store_row64_or_zero(tV + lane, dst + vcol, 1.0f, kr < a.seq && !on, kr < n);
      if (ws_.far && kb == 0) {
        float* part = ws_.base + ((static_cast<int64_t>(b) * a.kv_heads + kvh) * a.sinks + r) * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // dV | dK
          float x[32];
          ld_row32((c < 2 ? tV : tK) + lane + 32 * (c & 1), x);
          if (on) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) store8(part + 32 * c + i, x + i);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// One launch for both kinds, the dK/dV CTAs first (they have more to do).
template <int MODE>
__global__ void __maxnreg__(168) attn_window_bwd_kernel(const __grid_constant__ CUtensorMap tq64,
                                                        const __grid_constant__ CUtensorMap tq128,
                                                        const __grid_constant__ CUtensorMap td64,
                                                        const __grid_constant__ CUtensorMap td128,
                                                        const __grid_constant__ WindowArgs a,
                                                        const __grid_constant__ WindowScratch ws_,
                                                        __nv_bfloat16* __restrict__ dqkv, int n_dkv, int* err) {
  extern __shared__ __align__(1024) uint8_t sm[];
  if (reinterpret_cast<uintptr_t>(sm) & 1023u) {
    if (threadIdx.x == 0) atomicExch(err, DERR_ALIGN);
    return;
  }
  const int x = static_cast<int>(blockIdx.x);
  if (x < n_dkv)
    window_bwd_dkv<MODE>(a, &tq64, &tq128, &td64, ws_, dqkv, x, err, sm);
  else
    window_bwd_dq<MODE>(a, &tq64, &tq128, &td128, ws_, dqkv, x - n_dkv, err, sm);
}

// Blocks 0 .. n_sink-1: one sink key of one (sequence, key/value head); thread c
// adds column c of its dV | dK over the query blocks far from it, in order.
// Blocks n_sink ..: dtable of one head, added over (sequence, query block).
__global__ void __launch_bounds__(128) attn_window_finish_kernel(const __grid_constant__ WindowArgs a,
                                                                 const __grid_constant__ WindowScratch ws_,
                                                                 __nv_bfloat16* __restrict__ dqkv,
                                                                 float* __restrict__ dtable, int n_sink) {
  griddep_wait();
  griddep_launch();
  const int nqb = (a.seq + 127) / 128, c = threadIdx.x;
  int x = static_cast<int>(blockIdx.x);
  if (x < n_sink) {
    const int j = x % a.sinks, kvh = (x / a.sinks) % a.kv_heads, b = x / (a.sinks * a.kv_heads);
    const int n = seq_len(a, b);
    if (j >= n) return;
    const int group = a.heads / a.kv_heads, D = a.heads * HD;
    float v = ws_.base[((static_cast<int64_t>(b) * a.kv_heads + kvh) * a.sinks + j) * 128 + c];
    for (int g = 0; g < group; ++g) {
      const float* far = ws_.far + (static_cast<int64_t>(b) * a.heads + kvh * group + g) * nqb * a.sinks * 128;
#pragma unroll 8
      for (int qb = first_far_block(a.window); qb <= (n - 1) / 128; ++qb)
        v += far[(static_cast<int64_t>(qb) * a.sinks + j) * 128 + c];
    }
    const int64_t ld = static_cast<int64_t>(a.heads + 2 * a.kv_heads) * HD;
    __nv_bfloat16* dst = dqkv + (static_cast<int64_t>(b) * a.seq + j) * ld + D + kvh * HD;
    if (c < 64) dst[a.kv_heads * HD + c] = f2bf(v);
    else dst[c - 64] = f2bf(v * 0.125f);
    return;
  }
  const int h = x - n_sink;
  if (c >= a.ranks) return;
  double s = 0.0;
  const int64_t parts = static_cast<int64_t>(a.nseq) * nqb;
#pragma unroll 8
  for (int64_t p = 0; p < parts; ++p) s += ws_.tab[(p * a.heads + h) * a.ranks + c];
  dtable[static_cast<int64_t>(a.bucket[c]) * a.heads + h] += static_cast<float>(s);
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

// n^e >= md^k me^(e - k), in whole numbers of 32 words (4096^64 has 769 bits).
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
    a.start[a.ranks] = static_cast<int16_t>(starts[b]);
    a.bucket[a.ranks] = static_cast<uint8_t>(b);
    ++a.ranks;
  }
  a.last = a.start[a.ranks - 1];
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
  if (has_far(seq, window, sinks)) {
    const size_t s = sinks < seq ? sinks : seq;
    w.far = reinterpret_cast<float*>(take(nh * nqb * s * 128 * sizeof(float)));
    w.base = reinterpret_cast<float*>(take(nh * s * 128 * sizeof(float)));
  }
  if (ranks > 0) w.tab = reinterpret_cast<float*>(take(nh * nqb * ranks * sizeof(float)));
  w.bytes = off;
  return w;
}

int fwd_smem(const WindowArgs& a) { return FWD_LUT + (a.ranks ? lut_words(a.last) * 4 : 0); }
int bwd_smem(const WindowArgs& a, bool grad) {
  int s = BWD_LUT + (a.ranks ? lut_words(a.last) * 4 : 0);
  if (grad) s += 2 * a.ranks * 128 * 4 + (a.last / 32 + 1) * 4;
  return s;
}

int prepare_attention_window() {
  static std::atomic<unsigned long long> done{0};
  return once_per_device(done, []() -> int {
    constexpr int most = 227 * 1024;
    auto set = [](const void* f) {
      return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    };
    const void* all[] = {reinterpret_cast<const void*>(attn_window_fwd_kernel<false>),
                         reinterpret_cast<const void*>(attn_window_fwd_kernel<true>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<0>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<1>),
                         reinterpret_cast<const void*>(attn_window_bwd_kernel<2>)};
    for (const void* f : all)
      if (set(f) != cudaSuccess) return set_error(GPIPE_ERR_CUDA, "attention_window: shared-memory attribute failed");
    if (!encode_fn()) return set_error(GPIPE_ERR_CUDA, "attention_window: cuTensorMapEncodeTiled entry point not found");
    return static_cast<int>(GPIPE_OK);
  });
}

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
  rc = prepare_attention_window();
  if (rc) return rc;
  int* err = device_error_ptr();
  if (!err) return set_error(GPIPE_ERR_CUDA, "attention_window_fwd: no device error word");
  CUtensorMap tq;
  if (!make_tmap(&tq, qkv, static_cast<int64_t>(heads + 2 * kv_heads) * HD, seq, nseq, 128))
    return set_error(GPIPE_ERR_CUDA, "attention_window_fwd: tensor map creation failed");
  const int grid = ((seq + 127) / 128) * heads * nseq;
  (void)launch_k<true>(a.ranks ? attn_window_fwd_kernel<true> : attn_window_fwd_kernel<false>, grid, WIN_THREADS,
                       fwd_smem(a), s, tq, a, static_cast<__nv_bfloat16*>(o), lse, err);
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
  if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u))
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_bwd: scratch must be 256-B aligned");
  if (dtable_acc && !table)
    return set_error(GPIPE_ERR_INVALID_ARG, "attention_window_bwd: a table gradient needs the table");
  rc = prepare_attention_window();
  if (rc) return rc;
  int* err = device_error_ptr();
  if (!err) return set_error(GPIPE_ERR_CUDA, "attention_window_bwd: no device error word");
  const int64_t cols = static_cast<int64_t>(heads + 2 * kv_heads) * HD, D = static_cast<int64_t>(heads) * HD;
  CUtensorMap tq64, tq128, td64, td128;
  if (!make_tmap(&tq64, qkv, cols, seq, nseq, 64) || !make_tmap(&tq128, qkv, cols, seq, nseq, 128) ||
      !make_tmap(&td64, dout, D, seq, nseq, 64) || !make_tmap(&td128, dout, D, seq, nseq, 128))
    return set_error(GPIPE_ERR_CUDA, "attention_window_bwd: tensor map creation failed");
  const WindowScratch w = window_scratch(scratch, nseq, seq, heads, window, sinks, dtable_acc ? a.ranks : 0);
  const int64_t prep = static_cast<int64_t>(nseq) * pad128(seq) * heads * 8;
  (void)launch_k(attn_window_prep_kernel, static_cast<unsigned>((prep + 255) / 256), 256, 0, s, a,
                 static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, w.ld);
  rc = check_launch("attention_window_bwd (prep)");
  if (rc) return rc;
  const int nqb = (seq + 127) / 128, n_dkv = nqb * kv_heads * nseq, n_dq = nqb * heads * nseq;
  auto kern = dtable_acc ? attn_window_bwd_kernel<2> : (a.ranks ? attn_window_bwd_kernel<1> : attn_window_bwd_kernel<0>);
  (void)launch_k<true>(kern, n_dkv + n_dq, WIN_THREADS, bwd_smem(a, dtable_acc != nullptr), s, tq64, tq128, td64, td128,
                       a, w, static_cast<__nv_bfloat16*>(dqkv), n_dkv, err);
  rc = check_launch("attention_window_bwd");
  if (rc) return rc;
  const int n_sink = w.far ? nseq * kv_heads * a.sinks : 0;
  if (n_sink || dtable_acc) {
    (void)launch_k(attn_window_finish_kernel, n_sink + (dtable_acc ? heads : 0), 128, 0, s, a, w,
                   static_cast<__nv_bfloat16*>(dqkv), dtable_acc, n_sink);
    rc = check_launch("attention_window_bwd (finish)");
  }
  return rc;
}

}  // namespace gp
