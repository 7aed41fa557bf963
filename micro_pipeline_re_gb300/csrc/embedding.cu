// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   x_r = scale E[token_r],      dE[v] += scale sum_{r : token_r = v} dx_r
//
// The gradient first sorts the rows by token, stably, so that the rows of one
// token follow each other in ascending r (negative tokens and, after setting the
// error flag, tokens of vocab or more get the key vocab and end up behind the
// rest).  The sorted positions are cut into runs of 8 or 64; a group of threads
// reads a run's rows one after the other, many in flight, and sums them by token in
// order.  A token whose rows lie in one run is added to dE there; one that crosses
// runs leaves a sum in each, which a last kernel adds in order (more than 16 of them in
// eighths first) and then to dE.  So a frequent token's rows are read by many CTAs at once,
// and yet no sum depends on which of them was first.  Every element of dE receives one
// addition a call (a reduction in the L2: nobody waits for the old value).
//
// Few rows are not sorted: one launch finds each token's rows and adds them in quarters.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/gpipe.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_util.cuh"

namespace gp {
namespace {

// (times on the GPU, rows of 1024 columns)
// Sorted positions of a run: short ones of few rows, for CTAs enough, long ones of many, for
// fewer tokens that cross them.  24000 rows of text 38 us short, 32768 57 short and 46 long,
// 131072 157 with runs of 32 and 139 with 64.
constexpr int kShortRun = 8;
constexpr int kLongRun = 64;
constexpr int kLongRows = 24576;
// Rows up to which one launch does all: 256 rows 2.6 us, or 6.6 where all have one token; 257
// rows in three launches 5.3 us.
constexpr int kFewRows = 256;
// Rows up to which positions are counted by comparison: 2048 rows 9.5 us, sorted digit by digit
// 15; 4096 15.2 and 19.8; 8192 33.5 and 22.7.
constexpr int kRankRows = 4096;
constexpr int kDigit = 9;        // bits of a radix pass
constexpr int kBins = 1 << kDigit;
constexpr int kScatterThreads = 512;
constexpr int kTile = 512;       // positions of a CTA of a radix pass, at least
// And its CTAs, at most; up to kHalfRows rows half of them, since each reads all counts
// (131072 rows of 8 columns 41 us with 64, 44 with 128).
constexpr int kSortCtas = 128;
constexpr int kHalfRows = 1 << 18;
constexpr int kManyRuns = 16;  // more runs than these have a token's sums joined by several CTAs
constexpr int kJoinCtas = 8;   // join CTAs launched an SM, at most (6 at once)

// ---------------------------------------------------------------------------
// Lookup: a warp per row, 8 elements a lane and step; the product is rounded to
// fp32 and, for bf16 rows, once more.  2048 rows of 1024 columns, 4 MB in and 8 MB out, take
// 5 us from cold, a launch and one latency; a call takes the host about as long.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) embed_scaled_kernel(int rows, int d, int vocab,
                                                           const int32_t* __restrict__ tokens,
                                                           const __nv_bfloat16* __restrict__ emb, float scale,
                                                           T* __restrict__ x, int64_t ldx, int* err) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= rows) return;
  const int tok = tokens[r];
  const bool live = tok >= 0 && tok < vocab;
  if (tok >= vocab && lane == 0) atomicExch(err, DERR_BAD_TOKEN);
  const __nv_bfloat16* src = emb + static_cast<int64_t>(live ? tok : 0) * d;
  T* dst = x + static_cast<int64_t>(r) * ldx;
#pragma unroll 4
  for (int c = lane * 8; c < d; c += 256) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) load8(src + c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = live ? __fmul_rn(v[j], scale) : 0.f;
    store8(dst + c, v);
  }
}

// ---------------------------------------------------------------------------
// Sorting
// ---------------------------------------------------------------------------
__device__ __forceinline__ int key_of(int tok, int vocab) { return tok >= 0 && tok < vocab ? tok : vocab; }

// Few rows: row i's position is the number of rows with a smaller key, or the same
// one before it.  A CTA takes all keys into shared memory and ranks 32 rows, a lane
// each; its 8 warps compare them with an eighth of the keys each, which grows with the
// square of the rows (figures at kRankRows).
__global__ void __launch_bounds__(256) embed_rank_kernel(int rows, int vocab, const int32_t* __restrict__ tokens,
                                                         int* __restrict__ keys, int* __restrict__ order,
                                                         int* __restrict__ joins, int* err) {
  griddep_wait();
  griddep_launch();
  __shared__ __align__(16) int all[kRankRows];
  __shared__ int part[8][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * 32, i = row0 + lane;
  const int padded = (rows + 31) & ~31;
  if (blockIdx.x == 0 && tid < 2) joins[tid] = 0;
  bool bad = false;
#pragma unroll 8
  for (int j = tid; j < padded; j += 256) {
    const int tok = j < rows ? tokens[j] : -1;
    bad |= tok >= vocab;
    all[j] = j < rows ? key_of(tok, vocab) : vocab + 1;  // behind everything
  }
  if (bad && blockIdx.x == 0) atomicExch(err, DERR_BAD_TOKEN);
  __syncthreads();
  const int k = all[i];
  const int per = (padded / 32 + 7) / 8 * 32;  // of a warp
  const int j0 = warp * per, j1 = min(padded, j0 + per);
  int n = 0;
  // keys of earlier rows count when they are equal, too
  for (int j = j0; j < j1; j += 32) {
    const int4* t = reinterpret_cast<const int4*>(all + j);
    if (j == row0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n += t[e].x < k + (4 * e < lane) ? 1 : 0;
        n += t[e].y < k + (4 * e + 1 < lane) ? 1 : 0;
        n += t[e].z < k + (4 * e + 2 < lane) ? 1 : 0;
        n += t[e].w < k + (4 * e + 3 < lane) ? 1 : 0;
      }
    } else {
      const int below = k + (j < row0 ? 1 : 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n += t[e].x < below ? 1 : 0;
        n += t[e].y < below ? 1 : 0;
        n += t[e].z < below ? 1 : 0;
        n += t[e].w < below ? 1 : 0;
      }
    }
  }
  part[warp][lane] = n;
  __syncthreads();
  if (warp == 0 && i < rows) {
    int at = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) at += part[w][lane];
    keys[at] = k;
    order[at] = i;
  }
}

// Many rows: passes of kDigit bits from the lowest, each bound by its chain of latencies
// (131072 rows: 4 us to count, 11 and 8 for the two passes).  CTA c has `per` positions
// from c * per on; counts[c][bin] of the first pass, and zeros for the others'.
__global__ void __launch_bounds__(256) embed_count_kernel(int rows, int per, int vocab, int passes,
                                                          const int32_t* __restrict__ tokens, int* __restrict__ counts,
                                                          int* __restrict__ joins, int* err) {
  griddep_wait();
  griddep_launch();
  __shared__ int bins[kBins];
  for (int b = threadIdx.x; b < kBins; b += 256) bins[b] = 0;
  if (blockIdx.x == 0 && threadIdx.x < 2) joins[threadIdx.x] = 0;
  for (int p = 1; p < passes; ++p)
    for (int b = threadIdx.x; b < kBins; b += 256) counts[(p * kSortCtas + blockIdx.x) * kBins + b] = 0;
  __syncthreads();
  const int i0 = blockIdx.x * per, i1 = min(rows, i0 + per);
#pragma unroll 4
  for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += 256) {
    const int tok = tokens[i];
    if (tok >= vocab) atomicExch(err, DERR_BAD_TOKEN);
    atomicAdd(&bins[key_of(tok, vocab) & (kBins - 1)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < kBins; b += 256) counts[blockIdx.x * kBins + b] = bins[b];
}

// Its keys to their places: behind all smaller digits, the same digit of earlier
// CTAs and, in the CTA, of earlier warps (a warp has per / 16 consecutive positions)
// and earlier lanes.  A warp's first 128 keys are read once, ahead of everything.  The
// next pass's counts (of whole numbers, so in any order) are made as the keys land.
__global__ void __launch_bounds__(kScatterThreads) embed_scatter_kernel(
    int rows, int per, int vocab, int shift, bool first, const int* __restrict__ src,
    const int* __restrict__ src_order, const int* __restrict__ counts, int* __restrict__ next_counts,
    int* __restrict__ keys, int* __restrict__ order) {
  griddep_wait();
  griddep_launch();
  constexpr int kWarps = kScatterThreads / 32;
  static_assert(kScatterThreads == kBins, "thread t looks after bin t");
  __shared__ int at[kWarps][kBins], total[kBins], prior[kBins];
  __shared__ int wsum[kWarps];
  constexpr int kOnce = 4;  // keys a lane keeps
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = per / kWarps;
  const int i0 = blockIdx.x * per + warp * seg, i1 = min(min(rows, static_cast<int>(blockIdx.x + 1) * per), i0 + seg);
  auto key_at = [&](int i) { return i < i1 ? key_of(src[i], first ? vocab : INT32_MAX) : -1; };
  auto row_at = [&](int i) { return i < i1 ? (src_order ? src_order[i] : i) : 0; };
  int kept[kOnce], rows_kept[kOnce];
#pragma unroll
  for (int e = 0; e < kOnce; ++e) {
    kept[e] = key_at(i0 + 32 * e + lane);
    rows_kept[e] = row_at(i0 + 32 * e + lane);
  }
  // totals and those of earlier CTAs: a warp takes a sixteenth of the CTAs, a lane 16 bins
  {
    int4 all[4], earlier[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) all[u] = earlier[u] = make_int4(0, 0, 0, 0);
#pragma unroll 4
    for (int c = warp; c < static_cast<int>(gridDim.x); c += kWarps) {
      const int in = c < static_cast<int>(blockIdx.x) ? ~0 : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int4 n = *reinterpret_cast<const int4*>(counts + c * kBins + u * 128 + lane * 4);
        all[u].x += n.x;
        all[u].y += n.y;
        all[u].z += n.z;
        all[u].w += n.w;
        earlier[u].x += n.x & in;
        earlier[u].y += n.y & in;
        earlier[u].z += n.z & in;
        earlier[u].w += n.w & in;
      }
    }
    total[tid] = 0;
    prior[tid] = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) at[w][tid] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int b = u * 128 + lane * 4;
      const int4 n = all[u], e = earlier[u];
      const int nn[4] = {n.x, n.y, n.z, n.w}, ee[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (nn[j]) atomicAdd(&total[b + j], nn[j]);
        if (ee[j]) atomicAdd(&prior[b + j], ee[j]);
      }
    }
  }
  // the warps' counts, 32 keys at a time
  auto count = [&](int k) {
    const int bin = k < 0 ? kBins : (k >> shift) & (kBins - 1);
    const unsigned same = __match_any_sync(0xffffffffu, bin);
    if (bin < kBins && lane == __ffs(same) - 1) at[warp][bin] += __popc(same);
    __syncwarp();
  };
#pragma unroll
  for (int e = 0; e < kOnce; ++e)
    if (32 * e < seg) count(kept[e]);
  for (int i = i0 + 32 * kOnce; i < i1; i += 32) count(key_at(i + lane));
  __syncthreads();
  const int mine = total[tid];
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) wsum[warp] = sum;
  __syncthreads();
  int next = sum - mine + prior[tid];
  for (int w = 0; w < warp; ++w) next += wsum[w];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int n = at[w][tid];
    at[w][tid] = next;
    next += n;
  }
  __syncthreads();
  auto place = [&](int k, int row) {
    const int bin = k < 0 ? kBins : (k >> shift) & (kBins - 1);
    const unsigned same = __match_any_sync(0xffffffffu, bin);
    int to = 0;
    if (k >= 0) to = at[warp][bin] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (k >= 0 && lane == __ffs(same) - 1) at[warp][bin] += __popc(same);
    __syncwarp();
    if (k >= 0) {
      keys[to] = k;
      order[to] = row;
      if (next_counts)
        atomicAdd(next_counts + static_cast<int64_t>(to / per) * kBins + ((k >> (shift + kDigit)) & (kBins - 1)), 1);
    }
  };
#pragma unroll
  for (int e = 0; e < kOnce; ++e)
    if (32 * e < seg) place(kept[e], rows_kept[e]);
  for (int i = i0 + 32 * kOnce; i < i1; i += 32) place(key_at(i + lane), row_at(i + lane));
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------
// A thread's columns: 16 bytes of a row.
template <typename T> struct Cols;
template <> struct Cols<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint4 load(const float* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
  static __device__ __forceinline__ void add(float* a, uint4 u) {
    a[0] += __uint_as_float(u.x);
    a[1] += __uint_as_float(u.y);
    a[2] += __uint_as_float(u.z);
    a[3] += __uint_as_float(u.w);
  }
};
template <> struct Cols<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ uint4 load(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  }
  static __device__ __forceinline__ void add(float* a, uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_bf16x2(w[j]);
      a[2 * j] += f.x;
      a[2 * j + 1] += f.y;
    }
  }
};
// dE += v, an element's one addition of the call, always by the L2's reduction: a load, a
// multiply-add and a store would round the scaled sum with the addition and keep subnormals,
// where the others round it first and have them as zero.
__device__ __forceinline__ void add_to(float* p, float a, float b, float c, float d) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void add_to(float* p, float a) {
  asm volatile("red.global.add.f32 [%0], %1;" ::"l"(p), "f"(a) : "memory");
}

// Up to kFewRows rows in one launch: CTA (r, y) sums 64 threads' columns of the rows of
// token_r, if r is its first; its four groups of threads a quarter of the rows each.
template <typename T>
__global__ void __launch_bounds__(256) embed_few_kernel(int rows, int d, int vocab, const int32_t* __restrict__ tokens,
                                                        const T* __restrict__ dx, int64_t lddx, float scale,
                                                        float* __restrict__ demb, int* err) {
  griddep_wait();
  griddep_launch();
  using C = Cols<T>;
  __shared__ int mine[kFewRows];
  __shared__ int wcount[8];
  __shared__ __align__(16) float part[3][64 * C::N];
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k = tokens[r];
  const int t = tid < rows ? tokens[tid] : -1;
  if (k >= vocab && tid == 0) atomicExch(err, DERR_BAD_TOKEN);
  const bool same = t == k && tid < rows;
  if (__syncthreads_or(same && tid < r) || k < 0 || k >= vocab) return;
  const unsigned votes = __ballot_sync(0xffffffffu, same);
  if (lane == 0) wcount[warp] = __popc(votes);
  __syncthreads();
  int off = 0, n = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) off += wcount[w];
    n += wcount[w];
  }
  if (same) mine[off + __popc(votes & ((1u << lane) - 1u))] = tid;
  __syncthreads();
  const int group = tid >> 6, at = (tid & 63) * C::N, c = static_cast<int>(blockIdx.y) * 64 * C::N + at;
  const int per = (n + 3) / 4, i1 = min(n, (group + 1) * per);
  float acc[C::N] = {};
  if (c < d) {
#pragma unroll 8
    for (int i = group * per; i < i1; ++i) C::add(acc, C::load(dx + static_cast<int64_t>(mine[i]) * lddx + c));
  }
  if (group > 0) {
#pragma unroll
    for (int j = 0; j < C::N; ++j) part[group - 1][at + j] = acc[j];
  }
  if (n > 1) __syncthreads();
  if (group > 0 || c >= d) return;
  float* out = demb + static_cast<int64_t>(k) * d + c;
#pragma unroll
  for (int j = 0; j < C::N; ++j) {
    if (n > 1) acc[j] += part[0][at + j];
    if (n > 2) acc[j] += part[1][at + j];
    if (n > 3) acc[j] += part[2][at + j];
  }
#pragma unroll
  for (int j = 0; j < C::N; j += 4)
    add_to(out + j, scale * acc[j], scale * acc[j + 1], scale * acc[j + 2], scale * acc[j + 3]);
}

// Group y of the CTA: the run of sorted positions from p0 on; blockDim.x threads of 16
// bytes of a row each, and a slab of the columns for every blockIdx.y.  partial[run][2][d]:
// slot 0 the token that comes into the run or starts it and goes on behind it, slot 1 one
// that starts later and goes on.  The run in which such a token starts is put on a
// list: joins[2 + i] for i < joins[0], or for many runs joins[1 + runs - i] for i < joins[1].
// Bound by memory: 131072 rows of 1024 columns in fp32, 32000 tokens (702 MB with dE read and
// written) 110 us, 6.4 TB/s, where a read of dE before each addition took 273.
template <typename T, int RUN>
__global__ void __launch_bounds__(256) embed_sum_kernel(int rows, int d, int vocab, const int* __restrict__ keys,
                                                        const int* __restrict__ order, const T* __restrict__ dx,
                                                        int64_t lddx, float scale, float* __restrict__ demb,
                                                        float* __restrict__ partial, int* __restrict__ joins) {
  griddep_wait();
  griddep_launch();
  using C = Cols<T>;
  const int run = blockIdx.x * blockDim.y + threadIdx.y, p0 = run * RUN;
  if (p0 >= rows) return;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * C::N;
  if (c >= d) return;
  const int n = min(RUN, rows - p0);
  // the key before the run and the one behind it (-1: none)
  const int prev = p0 > 0 ? keys[p0 - 1] : -1, behind = p0 + RUN < rows ? keys[p0 + RUN] : -1;
  float acc[C::N] = {};
  int k = keys[p0];
  bool first = true;  // k is the run's first token
  auto flush = [&](bool goes_on) {
    if (k < vocab) {
      if (goes_on || (first && prev == k)) {
        float* out = partial + (static_cast<int64_t>(run) * 2 + (first ? 0 : 1)) * d + c;
#pragma unroll
        for (int j = 0; j < C::N; j += 4)
          *reinterpret_cast<float4*>(out + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        if (c == 0 && !(first && prev == k)) {
          const int64_t far = p0 + static_cast<int64_t>(kManyRuns) * RUN;
          if (far < rows && keys[far] == k) joins[1 + (rows + RUN - 1) / RUN - atomicAdd(joins + 1, 1)] = run;
          else joins[2 + atomicAdd(joins, 1)] = run;
        }
      } else {
        float* out = demb + static_cast<int64_t>(k) * d + c;
#pragma unroll
        for (int j = 0; j < C::N; j += 4)
          add_to(out + j, scale * acc[j], scale * acc[j + 1], scale * acc[j + 2], scale * acc[j + 3]);
      }
    }
    first = false;
#pragma unroll
    for (int j = 0; j < C::N; ++j) acc[j] = 0.f;
  };
#pragma unroll 1
  for (int q = 0; q < n; q += 8) {
    // (keys and order have room for a whole run behind the last row)
    const int4 ka = *reinterpret_cast<const int4*>(keys + p0 + q),
               kb = *reinterpret_cast<const int4*>(keys + p0 + q + 4);
    const int4 oa = *reinterpret_cast<const int4*>(order + p0 + q),
               ob = *reinterpret_cast<const int4*>(order + p0 + q + 4);
    const int kk[8] = {ka.x, ka.y, ka.z, ka.w, kb.x, kb.y, kb.z, kb.w};
    const int oo[8] = {oa.x, oa.y, oa.z, oa.w, ob.x, ob.y, ob.z, ob.w};
    uint4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (q + e < n && kk[e] < vocab) v[e] = C::load(dx + static_cast<int64_t>(oo[e]) * lddx + c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (q + e < n) {
        if (kk[e] != k) {
          flush(false);
          k = kk[e];
        }
        if (k < vocab) C::add(acc, v[e]);
      }
    }
  }
  flush(behind == k);
}

// The tokens that cross runs (131072 rows of text 10 us).  Those of up to kManyRuns runs take a CTA each, a warp for
// 128 columns, which adds the runs' sums in order.  The others take a CTA for every 128
// columns, whose warps add an eighth of the runs each, in order, and then those.
template <int RUN>
__global__ void __launch_bounds__(256, 6) embed_join_kernel(int rows, int d, const int* __restrict__ keys, float scale,
                                                         float* __restrict__ demb, const float* __restrict__ partial,
                                                         const int* __restrict__ joins) {
  griddep_wait();
  griddep_launch();
  __shared__ __align__(16) float part[8][128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto add_runs = [&](int b, bool whole, int j0, int j1, int c) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = j0; j < j1; ++j) {
      const int64_t slot = static_cast<int64_t>(b + j) * 2 + (j == 0 && !whole ? 1 : 0);
      const float4 v = *reinterpret_cast<const float4*>(partial + slot * d + c);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    return a;
  };
  const int many = joins[1], slabs = (d + 127) / 128, runs = (rows + RUN - 1) / RUN;
  // (from the last CTA on, as the others' first ones take longest)
  for (int64_t u = gridDim.x - 1 - blockIdx.x; u < static_cast<int64_t>(many) * slabs; u += gridDim.x) {
    const int b = joins[1 + runs - static_cast<int>(u / slabs)], c0 = static_cast<int>(u % slabs) * 128;
    const int next = (b + 1) * RUN;
    const int k = keys[next];
    const bool whole = keys[next - RUN] == k;
    int n = 2;
    for (bool more = true; more;) {
      const int64_t at = next + static_cast<int64_t>(n - 1 + tid) * RUN;
      const int found = __syncthreads_count(at < rows && keys[at] == k);
      n += found;
      more = found == 256;
    }
    const int per = (n + 7) / 8, c = c0 + lane * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < d) a = add_runs(b, whole, warp * per, min(n, (warp + 1) * per), c);
    *reinterpret_cast<float4*>(&part[warp][lane * 4]) = a;
    __syncthreads();
    if (tid < 128 && c0 + tid < d) {
      float t = part[0][tid];
#pragma unroll
      for (int w = 1; w < 8; ++w) t += part[w][tid];
      add_to(demb + static_cast<int64_t>(k) * d + c0 + tid, scale * t);
    }
    __syncthreads();
  }
  const int few = joins[0];
  for (int i = blockIdx.x; i < few; i += gridDim.x) {
    const int b = joins[2 + i];
    const int next = (b + 1) * RUN;  // the next run's first position, which has the token
    const int k = keys[next];
    const bool whole = keys[next - RUN] == k;  // slot 0 of its first run: it starts there
    int n = 2;                                 // its runs
#pragma unroll
    for (int e = 0; e < kManyRuns; e += 32) {
      const int64_t at = next + static_cast<int64_t>(1 + e + lane) * RUN;
      n += __popc(__ballot_sync(0xffffffffu, at < rows && keys[at] == k));
    }
    for (int c = warp * 128 + lane * 4; c < d; c += 1024) {
      const float4 a = add_runs(b, whole, 0, n, c);
      add_to(demb + static_cast<int64_t>(k) * d + c, scale * a.x, scale * a.y, scale * a.z, scale * a.w);
    }
  }
}

// Scratch: keys and order (two of each, for the passes, with room for a run behind
// them), counts, the list of tokens to join, partial sums.
struct SortScratch {
  size_t keys[2], order[2], counts, joins, partial, bytes;
  int run, runs;
};
SortScratch sort_scratch(int rows, int d) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  SortScratch s;
  s.run = rows <= kLongRows ? kShortRun : kLongRun;
  s.runs = (rows + s.run - 1) / s.run;
  const size_t n = up((static_cast<size_t>(rows) + kLongRun) * 4);
  size_t at = 0;
  for (int i = 0; i < 2; ++i) {
    s.keys[i] = at;
    s.order[i] = at + n;
    at += 2 * n;
  }
  s.counts = at;
  at += static_cast<size_t>(4 * kSortCtas) * kBins * 4;  // of up to four passes
  s.joins = at;
  at += up((static_cast<size_t>(s.runs) + 2) * 4);
  s.partial = at;
  at += up(static_cast<size_t>(s.runs) * 2 * d * 4);
  s.bytes = at;
  return s;
}

int check(const char* what) {
  count_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(GPIPE_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return GPIPE_OK;
}

bool sizes_ok(int rows, int d, int vocab) {
  return rows >= 1 && rows <= (1 << 27) && d >= 8 && d <= (1 << 16) && d % 8 == 0 && vocab >= 1 && vocab <= (1 << 30);
}
constexpr const char* kSizes = "need 1 <= rows <= 2^27, 8 <= d <= 2^16, d % 8 == 0 and 1 <= vocab <= 2^30";

}  // namespace

int launch_embedding_scaled_fwd(int dtype, int rows, int d, int vocab, const int32_t* tokens, const void* emb,
                                float scale, void* x, int64_t ldx, cudaStream_t s) {
  using attn::al16;
  using attn::Range;
  if (dtype != DT_F32 && dtype != DT_BF16)
    return set_error(GPIPE_ERR_UNSUPPORTED, "embedding_scaled_fwd: dtype must be 0 or 1");
  if (!sizes_ok(rows, d, vocab)) return set_error(GPIPE_ERR_INVALID_ARG, "embedding_scaled_fwd: %s", kSizes);
  if (!(scale > -INFINITY && scale < INFINITY))
    return set_error(GPIPE_ERR_INVALID_ARG, "embedding_scaled_fwd: the scale must be finite");
  if (!tokens || !attn::al4(tokens) || !emb || !al16(emb) || !x || !al16(x) || ldx < d || ldx % 8)
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "embedding_scaled_fwd: need tokens, 16-B aligned emb and x, and ldx >= d a multiple of 8");
  const size_t es = dtype == DT_F32 ? 4 : 2;
  const Range out = {x, (static_cast<size_t>(rows - 1) * ldx + d) * es};
  if (overlaps(out, {Range{tokens, static_cast<size_t>(rows) * 4}, Range{emb, static_cast<size_t>(vocab) * d * 2}}))
    return set_error(GPIPE_ERR_INVALID_ARG, "embedding_scaled_fwd: x overlaps an input");
  int* err = device_error_ptr();
  if (!err) return set_error(GPIPE_ERR_CUDA, "embedding_scaled_fwd: no device error word");
  const auto* e = static_cast<const __nv_bfloat16*>(emb);
  const int ctas = (rows + 7) / 8;
  if (dtype == DT_F32)
    (void)launch_k(embed_scaled_kernel<float>, ctas, 256, 0, s, rows, d, vocab, tokens, e, scale,
                   static_cast<float*>(x), ldx, err);
  else
    (void)launch_k(embed_scaled_kernel<__nv_bfloat16>, ctas, 256, 0, s, rows, d, vocab, tokens, e, scale,
                   static_cast<__nv_bfloat16*>(x), ldx, err);
  return check("embedding_scaled_fwd");
}

size_t embedding_sorted_bwd_scratch_bytes(int rows, int d, int vocab) {
  return sizes_ok(rows, d, vocab) ? sort_scratch(rows, d).bytes : 0;
}

int launch_embedding_sorted_bwd(int dtype, int rows, int d, int vocab, const int32_t* tokens, const void* dx,
                                int64_t lddx, float scale, float* demb, void* scratch, cudaStream_t s) {
  using attn::al16;
  using attn::Range;
  if (dtype != DT_F32 && dtype != DT_BF16)
    return set_error(GPIPE_ERR_UNSUPPORTED, "embedding_sorted_bwd: dtype must be 0 or 1");
  if (!sizes_ok(rows, d, vocab)) return set_error(GPIPE_ERR_INVALID_ARG, "embedding_sorted_bwd: %s", kSizes);
  if (!(scale > -INFINITY && scale < INFINITY))
    return set_error(GPIPE_ERR_INVALID_ARG, "embedding_sorted_bwd: the scale must be finite");
  if (!tokens || !attn::al4(tokens) || !dx || !al16(dx) || !demb || !al16(demb) || lddx < d || lddx % 8)
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "embedding_sorted_bwd: need tokens, 16-B aligned dx and demb, and lddx >= d a multiple of 8");
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256)
    return set_error(GPIPE_ERR_INVALID_ARG, "embedding_sorted_bwd: scratch must be 256-B aligned");
  const SortScratch at = sort_scratch(rows, d);
  const size_t es = dtype == DT_F32 ? 4 : 2;
  const Range tok = {tokens, static_cast<size_t>(rows) * 4},
              in = {dx, (static_cast<size_t>(rows - 1) * lddx + d) * es},
              out = {demb, static_cast<size_t>(vocab) * d * 4}, work = {scratch, at.bytes};
  if (overlaps(out, {tok, in, work}) || overlaps(work, {tok, in}))
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "embedding_sorted_bwd: demb and scratch may overlap neither each other nor the inputs");
  int* err = device_error_ptr();
  if (!err) return set_error(GPIPE_ERR_CUDA, "embedding_sorted_bwd: no device error word");
  auto sums = [&](auto* in_rows) -> int {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(in_rows)>>;
    if (rows <= kFewRows) {
      const int wide = 64 * Cols<T>::N;
      (void)launch_k(embed_few_kernel<T>, dim3(rows, (d + wide - 1) / wide), 256, 0, s, rows, d, vocab, tokens,
                     in_rows, lddx, scale, demb, err);
      return check("embedding_sorted_bwd");
    }
    char* w = static_cast<char*>(scratch);
    int* keys[2] = {reinterpret_cast<int*>(w + at.keys[0]), reinterpret_cast<int*>(w + at.keys[1])};
    int* order[2] = {reinterpret_cast<int*>(w + at.order[0]), reinterpret_cast<int*>(w + at.order[1])};
    int* counts = reinterpret_cast<int*>(w + at.counts);
    int* joins = reinterpret_cast<int*>(w + at.joins);
    float* partial = reinterpret_cast<float*>(w + at.partial);
    int have = 0;
    if (rows <= kRankRows) {
      (void)launch_k(embed_rank_kernel, (rows + 31) / 32, 256, 0, s, rows, vocab, tokens, keys[0], order[0], joins,
                     err);
      if (const int rc = check("embedding_sorted_bwd")) return rc;
    } else {
      int bits = 1;
      while (bits < 31 && (vocab >> bits) != 0) ++bits;  // keys 0 .. vocab
      const int ctas = std::min(rows <= kHalfRows ? kSortCtas / 2 : kSortCtas, (rows + kTile - 1) / kTile);
      const int per = ((rows + ctas - 1) / ctas + 511) / 512 * 512;
      const int grid = (rows + per - 1) / per;
      const int passes = (bits + kDigit - 1) / kDigit;
      (void)launch_k(embed_count_kernel, grid, 256, 0, s, rows, per, vocab, passes, tokens, counts, joins, err);
      if (const int rc = check("embedding_sorted_bwd")) return rc;
      const int* src = tokens;
      const int* src_order = nullptr;
      for (int p = 0; p < passes; ++p) {
        const int* now = counts + static_cast<int64_t>(p) * kSortCtas * kBins;
        int* then = p + 1 < passes ? counts + static_cast<int64_t>(p + 1) * kSortCtas * kBins : nullptr;
        have = p & 1;
        (void)launch_k(embed_scatter_kernel, grid, kScatterThreads, 0, s, rows, per, vocab, p * kDigit, p == 0, src,
                       src_order, now, then, keys[have], order[have]);
        if (const int rc = check("embedding_sorted_bwd")) return rc;
        src = keys[have];
        src_order = order[have];
      }
    }
    const int n = Cols<T>::N;
    int tx = 8;
    while (tx < 256 && tx * n < d) tx *= 2;
    const dim3 block(tx, 256 / tx);
    const dim3 grid((at.runs + block.y - 1) / block.y, (d + tx * n - 1) / (tx * n));
    const int* k = keys[have];
    const int* o = order[have];
    const bool few = at.run == kShortRun;
    (void)launch_k(few ? embed_sum_kernel<T, kShortRun> : embed_sum_kernel<T, kLongRun>, grid, block, 0, s, rows, d,
                   vocab, k, o, in_rows, lddx, scale, demb, partial, joins);
    if (const int rc = check("embedding_sorted_bwd")) return rc;
    const int join = std::min(at.runs, kJoinCtas * num_sms());
    (void)launch_k(few ? embed_join_kernel<kShortRun> : embed_join_kernel<kLongRun>, join, 256, 0, s, rows, d, k,
                   scale, demb, static_cast<const float*>(partial), static_cast<const int*>(joins));
    return check("embedding_sorted_bwd");
  };
  return dtype == DT_F32 ? sums(static_cast<const float*>(dx)) : sums(static_cast<const __nv_bfloat16*>(dx));
}

}  // namespace gp
