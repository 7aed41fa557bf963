// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   x_r = scale E[token_r],      dE[v] += scale sum_{r : token_r = v} dx_r
//
// The gradient first sorts the rows by token, stably, so that the rows of one
// token follow each other in ascending r (negative tokens and, after setting the
// error flag, tokens of vocab or more get the key vocab and end up behind the
// rest).  The sorted positions are cut at the starts of the tokens and at every
// kRun-th position; each piece is summed on its own, in order, and
//   - a piece that holds all rows of its token adds its sum to dE at once,
//   - the pieces of a longer token leave their sums in scratch, where a second
//     kernel adds them in order and then to dE.
// So a frequent token's rows are read by many CTAs at once, and yet no sum
// depends on which of them was first: no floating-point atomics.
#include <algorithm>
#include <cmath>

#include "../../include/gpipe.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_util.cuh"

namespace gp {
namespace {

constexpr int kRun = 32;         // sorted positions between two cuts
constexpr int kRankRows = 8192;  // rows up to which positions are counted by comparison
constexpr int kDigit = 9;        // bits of a radix pass
constexpr int kBins = 1 << kDigit;
constexpr int kSortCtas = 128;   // CTAs of a radix pass, at most

// ---------------------------------------------------------------------------
// Lookup: a warp per row, 8 elements a lane and step; the product is rounded to
// fp32 and, for bf16 rows, once more.
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
// one before it.  A CTA ranks 32 rows (a lane each); its 8 warps compare them with
// an eighth of the rows each.
__global__ void __launch_bounds__(256) embed_rank_kernel(int rows, int vocab, const int32_t* __restrict__ tokens,
                                                         int* __restrict__ keys, int* __restrict__ order, int* err) {
  griddep_wait();
  griddep_launch();
  __shared__ int part[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * 32, i = row0 + lane;
  const int tok = i < rows ? tokens[i] : -1;
  const int k = key_of(tok, vocab);
  if (warp == 0 && tok >= vocab) atomicExch(err, DERR_BAD_TOKEN);
  const int per = (rows + 7) / 8;
  const int j0 = warp * per, j1 = min(rows, j0 + per);
  int n = 0;
#pragma unroll 8
  for (int j = j0; j < j1; ++j) n += key_of(__ldg(tokens + j), vocab) < k + (j < i ? 1 : 0) ? 1 : 0;
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

// Many rows: passes of kDigit bits from the lowest.  CTA c has `per` positions
// from c * per on; counts[c][bin] of the pass.
__global__ void __launch_bounds__(256) embed_count_kernel(int rows, int per, int vocab, int shift, bool first,
                                                          const int* __restrict__ src, int* __restrict__ counts,
                                                          int* err) {
  griddep_wait();
  griddep_launch();
  __shared__ int bins[kBins];
  for (int b = threadIdx.x; b < kBins; b += 256) bins[b] = 0;
  __syncthreads();
  const int i0 = blockIdx.x * per, i1 = min(rows, i0 + per);
  for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += 256) {
    int k = src[i];
    if (first) {
      if (k >= vocab) atomicExch(err, DERR_BAD_TOKEN);
      k = key_of(k, vocab);
    }
    atomicAdd(&bins[(k >> shift) & (kBins - 1)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < kBins; b += 256) counts[blockIdx.x * kBins + b] = bins[b];
}

// Its keys to their places: behind all smaller digits, the same digit of earlier
// CTAs and, in the CTA, of earlier warps (a warp has per / 8 consecutive positions)
// and earlier lanes.
__global__ void __launch_bounds__(256) embed_scatter_kernel(int rows, int per, int vocab, int shift, bool first,
                                                            const int* __restrict__ src,
                                                            const int* __restrict__ src_order,
                                                            const int* __restrict__ counts, int* __restrict__ keys,
                                                            int* __restrict__ order) {
  griddep_wait();
  griddep_launch();
  __shared__ int at[8][kBins];
  __shared__ int wsum[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // thread t: bins 2t and 2t + 1, totals and those of earlier CTAs
  int total[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll 16
  for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
    const int2 n = *reinterpret_cast<const int2*>(counts + c * kBins + 2 * tid);
    total[0] += n.x;
    total[1] += n.y;
    if (c < static_cast<int>(blockIdx.x)) {
      before[0] += n.x;
      before[1] += n.y;
    }
  }
  int sum = total[0] + total[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) wsum[warp] = sum;
  for (int b = tid; b < 8 * kBins; b += 256) (&at[0][0])[b] = 0;
  __syncthreads();
  int base = sum - total[0] - total[1];
  for (int w = 0; w < warp; ++w) base += wsum[w];

  // the warps' counts
  const int seg = per / 8;
  const int i0 = blockIdx.x * per + warp * seg, i1 = min(min(rows, static_cast<int>(blockIdx.x + 1) * per), i0 + seg);
  for (int i = i0; i < i1; i += 32) {
    const int k = i + lane < i1 ? key_of(src[i + lane], first ? vocab : INT32_MAX) : -1;
    const int bin = k < 0 ? kBins : (k >> shift) & (kBins - 1);
    const unsigned same = __match_any_sync(0xffffffffu, bin);
    if (bin < kBins && lane == __ffs(same) - 1) at[warp][bin] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    int next = base + before[e] + (e ? total[0] : 0);
    for (int w = 0; w < 8; ++w) {
      const int n = at[w][2 * tid + e];
      at[w][2 * tid + e] = next;
      next += n;
    }
  }
  __syncthreads();
  for (int i = i0; i < i1; i += 32) {
    const bool mine = i + lane < i1;
    const int k = mine ? key_of(src[i + lane], first ? vocab : INT32_MAX) : -1;
    const int bin = k < 0 ? kBins : (k >> shift) & (kBins - 1);
    const unsigned same = __match_any_sync(0xffffffffu, bin);
    int to = 0;
    if (mine) to = at[warp][bin] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (mine && lane == __ffs(same) - 1) at[warp][bin] += __popc(same);
    __syncwarp();
    if (mine) {
      keys[to] = k;
      order[to] = src_order ? src_order[i + lane] : i + lane;
    }
  }
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------
// Group y of the CTA: the piece that starts at sorted position p, if one does.
// tx threads of 8 columns each walk over the row.  Scratch: partial[block][2][d],
// slot 0 the piece that starts the block, slot 1 the one that ends it.
template <typename T>
__global__ void __launch_bounds__(256) embed_sum_kernel(int rows, int d, int vocab, const int* __restrict__ keys,
                                                        const int* __restrict__ order, const T* __restrict__ dx,
                                                        int64_t lddx, float scale, float* __restrict__ demb,
                                                        float* __restrict__ partial) {
  griddep_wait();
  griddep_launch();
  const int p = blockIdx.x * blockDim.y + threadIdx.y;
  if (p >= rows) return;
  const int k = keys[p];
  const bool starts = p == 0 || keys[p - 1] != k;
  if (k >= vocab || !(starts || p % kRun == 0)) return;
  const int most = min(rows, (p / kRun + 1) * kRun);
  for (int c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
    float* out = demb + static_cast<int64_t>(k) * d + c;
    float old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (starts) load8(out, old);  // (of no use if the token goes on behind the piece)
    float acc[8];
    load8(dx + static_cast<int64_t>(order[p]) * lddx + c, acc);
    int q = p + 1;
    bool more = true;
    while (more && q < most) {
      constexpr int kAhead = 8;
      float v[kAhead][8];
      int n = 0;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        more = more && q + e < most && keys[q + e] == k;
        if (more) {
          load8(dx + static_cast<int64_t>(order[q + e]) * lddx + c, v[e]);
          ++n;
        }
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (e < n) {
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += v[e][j];
        }
      }
      q += n;
    }
    const bool ends = q == rows || keys[q] != k;
    if (starts && ends) {
#pragma unroll
      for (int j = 0; j < 8; ++j) old[j] = fmaf(scale, acc[j], old[j]);
      store8(out, old);
    } else {
      store8(partial + (static_cast<int64_t>(p / kRun) * 2 + (p % kRun ? 1 : 0)) * d + c, acc);
    }
  }
}

// A token whose rows cross a cut: CTA b has the one that starts in block b and goes
// on behind it.  Its blocks' sums are added by 8 warps, an eighth of the blocks
// each in order, then warp by warp.
__global__ void __launch_bounds__(256) embed_join_kernel(int rows, int d, int vocab, const int* __restrict__ keys,
                                                         float scale, float* __restrict__ demb,
                                                         const float* __restrict__ partial) {
  griddep_wait();
  griddep_launch();
  __shared__ int sh_end;
  __shared__ __align__(16) float part[8][128];
  const int b = blockIdx.x, last = (b + 1) * kRun - 1;
  if (last + 1 >= rows) return;
  const int k = keys[last];
  if (k >= vocab || keys[last + 1] != k) return;
  // does it start in this block?
  const int first = b * kRun;
  if (first > 0 && keys[first - 1] == k) return;
  const bool whole = keys[first] == k;  // it fills the block from its first position
  // the last block that has rows of it: the first position behind `last` with another key, by bisection
  if (threadIdx.x == 0) {
    int lo = last + 1, hi = rows;  // keys[lo] == k; keys[hi] != k or hi == rows
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (keys[mid] == k) lo = mid;
      else hi = mid;
    }
    sh_end = lo / kRun;
  }
  __syncthreads();
  const int n = sh_end - b;  // blocks behind this one
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (n + 1 + 7) / 8, j0 = warp * per, j1 = min(n + 1, j0 + per);
  const int64_t slot0 = static_cast<int64_t>(b) * 2;
  for (int c0 = blockIdx.y * 128; c0 < d; c0 += gridDim.y * 128) {
    const int c = c0 + lane * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < d) {
#pragma unroll 8
      for (int j = j0; j < j1; ++j) {
        const int64_t slot = j == 0 ? slot0 + (whole ? 0 : 1) : slot0 + 2 * j;
        const float4 v = *reinterpret_cast<const float4*>(partial + slot * d + c);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
    }
    *reinterpret_cast<float4*>(&part[warp][lane * 4]) = a;
    __syncthreads();
    const int e = c0 + static_cast<int>(threadIdx.x);
    if (threadIdx.x < 128 && e < d) {
      float t = part[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; ++w) t += part[w][threadIdx.x];
      float* out = demb + static_cast<int64_t>(k) * d + e;
      *out = fmaf(scale, t, *out);
    }
    __syncthreads();
  }
}

// Scratch: keys and order (two of each, for the passes), counts, partial sums.
struct SortScratch {
  size_t keys[2], order[2], counts, partial, bytes;
};
SortScratch sort_scratch(int rows, int d) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  SortScratch s;
  const size_t n = up(static_cast<size_t>(rows) * 4);
  size_t at = 0;
  for (int i = 0; i < 2; ++i) {
    s.keys[i] = at;
    s.order[i] = at + n;
    at += 2 * n;
  }
  s.counts = at;
  at += static_cast<size_t>(kSortCtas) * kBins * 4;
  s.partial = at;
  at += up((static_cast<size_t>(rows) + kRun - 1) / kRun * 2 * d * 4);
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
  char* w = static_cast<char*>(scratch);
  int* keys[2] = {reinterpret_cast<int*>(w + at.keys[0]), reinterpret_cast<int*>(w + at.keys[1])};
  int* order[2] = {reinterpret_cast<int*>(w + at.order[0]), reinterpret_cast<int*>(w + at.order[1])};
  int* counts = reinterpret_cast<int*>(w + at.counts);
  float* partial = reinterpret_cast<float*>(w + at.partial);
  int have = 0;
  if (rows <= kRankRows) {
    (void)launch_k(embed_rank_kernel, (rows + 31) / 32, 256, 0, s, rows, vocab, tokens, keys[0], order[0], err);
    if (const int rc = check("embedding_sorted_bwd")) return rc;
  } else {
    int bits = 1;
    while (bits < 31 && (vocab >> bits) != 0) ++bits;  // keys 0 .. vocab
    const int ctas = std::min(kSortCtas, (rows + 2047) / 2048);
    const int per = ((rows + ctas - 1) / ctas + 255) / 256 * 256;
    const int grid = (rows + per - 1) / per;
    const int* src = tokens;
    const int* src_order = nullptr;
    for (int shift = 0; shift < bits; shift += kDigit, have ^= 1) {
      const bool first = shift == 0;
      (void)launch_k(embed_count_kernel, grid, 256, 0, s, rows, per, vocab, shift, first, src, counts, err);
      if (const int rc = check("embedding_sorted_bwd")) return rc;
      (void)launch_k(embed_scatter_kernel, grid, 256, 0, s, rows, per, vocab, shift, first, src, src_order,
                     static_cast<const int*>(counts), keys[have], order[have]);
      if (const int rc = check("embedding_sorted_bwd")) return rc;
      src = keys[have];
      src_order = order[have];
    }
    have ^= 1;  // the last pass's
  }
  int tx = 8;
  while (tx < 128 && tx * 8 < d) tx *= 2;
  const dim3 block(tx, 256 / tx);
  const int groups = static_cast<int>((rows + block.y - 1) / block.y);
  const int* k = keys[have];
  const int* o = order[have];
  if (dtype == DT_F32)
    (void)launch_k(embed_sum_kernel<float>, groups, block, 0, s, rows, d, vocab, k, o, static_cast<const float*>(dx),
                   lddx, scale, demb, partial);
  else
    (void)launch_k(embed_sum_kernel<__nv_bfloat16>, groups, block, 0, s, rows, d, vocab, k, o,
                   static_cast<const __nv_bfloat16*>(dx), lddx, scale, demb, partial);
  if (const int rc = check("embedding_sorted_bwd")) return rc;
  if (rows <= kRun) return GPIPE_OK;  // no cut that a token could cross
  (void)launch_k(embed_join_kernel, dim3((rows - 1) / kRun, std::min(4, (d + 127) / 128)), 256, 0, s, rows, d, vocab,
                 k, scale, demb, static_cast<const float*>(partial));
  return check("embedding_sorted_bwd");
}

}  // namespace gp
