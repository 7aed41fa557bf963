// The head's loss without the logits: next-token cross-entropy of h E^T over the
// tied matrix E, and its gradients with respect to h and E, made for a piece of
// the vocabulary at a time.
//
//   z = h_r E^T (limited to [-clip, clip]),  m = max z,  s = sum e^{z - m}
//   loss_r = w_r a ((m - z_t) + ln s),       a = inv_count
//   g = w_r (e^{z - m} / s - onehot(t)),     dh = a g E,  dE = a g^T h
//
// Two passes over the vocabulary: the first leaves m, s and z_t of every row, the
// second makes a piece of z again, turns it into g (bf16) and multiplies that by E
// and by h.
#include <algorithm>
#include <cmath>

#include "../../include/gpipe.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_util.cuh"

namespace gp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct HeadRow {  // what the passes know of a row
  float m, s, zt, w;
};

struct HeadArgs {
  int rows, d, vocab, seq, row0;
  const int32_t* tokens;
  const float* weight;
  float inv_count, clip;
};

// Target of row r, or -1 (none: the end of a sequence, a negative id, weight 0).
__device__ __forceinline__ int head_target(const HeadArgs& a, int r, float& w, int* err) {
  w = a.weight ? a.weight[r] : 1.f;
  const int64_t at = static_cast<int64_t>(a.row0) + r;
  if (w == 0.f || at % a.seq == a.seq - 1) return -1;
  const int t = a.tokens[at + 1];
  if (t >= a.vocab && err) atomicExch(err, DERR_BAD_TOKEN);
  return t >= 0 && t < a.vocab ? t : -1;
}

__device__ __forceinline__ float limit(float z, float c) {  // keeps NaN
  if (c <= 0.f) return z;
  return z > c ? c : (z < -c ? -c : z);
}

// A warp per row: h with the rows of no target set to zero (they may hold anything).
__global__ void __launch_bounds__(256) head_rows_kernel(HeadArgs a, const __nv_bfloat16* __restrict__ h, int64_t ldh,
                                                        __nv_bfloat16* __restrict__ hm, HeadRow* __restrict__ info,
                                                        int* err) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.rows) return;
  float w;
  const int t = head_target(a, r, w, lane == 0 ? err : nullptr);
  for (int c = lane * 8; c < a.d; c += 256) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t >= 0) v = *reinterpret_cast<const uint4*>(h + r * ldh + c);
    *reinterpret_cast<uint4*>(hm + static_cast<int64_t>(r) * a.d + c) = v;
  }
  if (lane == 0) info[r] = HeadRow{-INFINITY, 0.f, 0.f, t >= 0 ? w : 0.f};
}

// A CTA per row: the piece's columns into m, s and z_t.
__global__ void __launch_bounds__(256) head_stats_kernel(HeadArgs a, const float* __restrict__ z, int64_t ldz, int v0,
                                                         int cols, HeadRow* __restrict__ info) {
  griddep_wait();
  griddep_launch();
  __shared__ float red[8];
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* zr = z + r * ldz;
  HeadRow row = info[r];
  float m = row.m;
  for (int c = tid; c < cols; c += 256) m = fmaxf(m, limit(zr[c], a.clip));
  m = warp_max(m);
  if (lane == 0) red[warp] = m;
  __syncthreads();
  for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
  __syncthreads();
  float s = 0.f;
  for (int c = tid; c < cols; c += 256) s += ex2_approx((limit(zr[c], a.clip) - m) * kLog2e);
  s = warp_sum(s);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (tid == 0) {
    s = row.s > 0.f ? row.s * ex2_approx((row.m - m) * kLog2e) : 0.f;
    for (int w = 0; w < 8; ++w) s += red[w];
    float w;
    const int t = head_target(a, r, w, nullptr);
    if (t >= v0 && t < v0 + cols) row.zt = limit(zr[t - v0], a.clip);
    info[r] = HeadRow{m, s, row.zt, row.w};
  }
}

__global__ void __launch_bounds__(256) head_loss_kernel(int rows, float inv_count, const HeadRow* __restrict__ info,
                                                        float* __restrict__ loss) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= rows) return;
  const HeadRow i = info[r];
  loss[r] = i.w != 0.f ? i.w * inv_count * ((i.m - i.zt) + logf(i.s)) : 0.f;
}

// A CTA per row: the piece of z into g (times inv_count), bf16.
__global__ void __launch_bounds__(256) head_grad_kernel(HeadArgs a, const float* __restrict__ z, int64_t ldz, int v0,
                                                        int cols, const HeadRow* __restrict__ info,
                                                        __nv_bfloat16* __restrict__ g) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x;
  const float* zr = z + r * ldz;
  const HeadRow i = info[r];
  float w;
  const int t = head_target(a, r, w, nullptr);
  const float wa = i.w * a.inv_count, inv_s = 1.f / i.s;
  for (int c = threadIdx.x; c < cols; c += 256) {
    float v = 0.f;
    if (t >= 0) {
      const float x = zr[c];
      v = wa * (ex2_approx((limit(x, a.clip) - i.m) * kLog2e) * inv_s - (v0 + c == t ? 1.f : 0.f));
      if (a.clip > 0.f && fabsf(x) > a.clip) v = 0.f;
    }
    g[r * ldz + c] = f2bf(v);
  }
}

__global__ void __launch_bounds__(256) head_dh_kernel(int rows, int d, const float* __restrict__ src,
                                                      __nv_bfloat16* __restrict__ dh, int64_t lddh) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= rows) return;
  for (int c = lane * 8; c < d; c += 256) {
    float v[8];
    load8(src + static_cast<int64_t>(r) * d + c, v);
    store8(dh + r * lddh + c, v);
  }
}

int check(const char* what) {
  count_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(GPIPE_ERR_CUDA, "head_loss: %s launch: %s", what, cudaGetErrorString(e));
  return GPIPE_OK;
}

bool sizes_ok(int rows, int d, int vocab, int piece) {
  return rows >= 1 && rows <= (1 << 24) && d >= 8 && d <= (1 << 16) && d % 8 == 0 && vocab >= 1 &&
         vocab <= (1 << 27) && piece >= 0;
}

// Columns of a piece: a multiple of 256; 0 asks for as many as make g 256 MB.
int piece_columns(int rows, int vocab, int piece) {
  int64_t p = piece ? piece : std::max<int64_t>(2048, (static_cast<int64_t>(1) << 27) / rows);
  p = std::min<int64_t>((p + 255) / 256 * 256, (static_cast<int64_t>(vocab) + 255) / 256 * 256);
  return static_cast<int>(p);
}

struct HeadScratch {
  size_t info, hm, z, g, dh, bytes;
};
HeadScratch head_scratch(int rows, int d, int piece, int grads) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  const size_t n = static_cast<size_t>(rows);
  HeadScratch s;
  s.info = 0;
  s.hm = up(n * sizeof(HeadRow));
  s.z = s.hm + up(n * d * 2);
  s.g = s.z + up(n * piece * 4);
  s.dh = s.g + (grads ? up(n * piece * 2) : 0);
  s.bytes = s.dh + (grads & 1 ? up(n * d * 4) : 0);
  return s;
}

}  // namespace

size_t head_loss_scratch_bytes(int rows, int d, int vocab, int piece, int grads) {
  if (!sizes_ok(rows, d, vocab, piece) || grads < 0 || grads > 3) return 0;
  return head_scratch(rows, d, piece_columns(rows, vocab, piece), grads).bytes;
}

int launch_head_loss(int rows, int d, int vocab, const void* h, int64_t ldh, const void* emb, int seq,
                     const int32_t* tokens, int row0, const float* row_weight, float inv_count, float clip, int piece,
                     float* loss_rows, void* dh, int64_t lddh, int demb_dtype, void* demb, void* scratch,
                     cudaStream_t st) {
  using attn::al16;
  using attn::al4;
  using attn::Range;
  if (!sizes_ok(rows, d, vocab, piece))
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "head_loss: need 1 <= rows <= 2^24, 8 <= d <= 2^16, d %% 8 == 0, 1 <= vocab <= 2^27 and piece >= 0");
  if (demb && demb_dtype != DT_F32 && demb_dtype != DT_BF16)
    return set_error(GPIPE_ERR_UNSUPPORTED, "head_loss: demb_dtype must be 0 or 1");
  if (seq < 1 || row0 < 0 || static_cast<int64_t>(row0) + rows >= INT32_MAX)
    return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: need seq >= 1, row0 >= 0 and row0 + rows < 2^31 - 1");
  if (!(inv_count > -INFINITY && inv_count < INFINITY) || !(clip >= 0.f && clip < INFINITY))
    return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: need a finite inv_count and a finite clip >= 0");
  if (!h || !al16(h) || !emb || !al16(emb) || ldh < d || ldh % 8)
    return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: need 16-B aligned h and emb, and ldh >= d a multiple of 8");
  if (!tokens || !al4(tokens) || !al4(row_weight) || !loss_rows || !al4(loss_rows))
    return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: need tokens and loss_rows, aligned to their elements");
  if (dh && (!al16(dh) || lddh < d || lddh % 8))
    return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: need a 16-B aligned dh and lddh >= d a multiple of 8");
  if (!al16(demb)) return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: demb must be 16-B aligned");
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256)
    return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: scratch must be 256-B aligned");
  const int grads = (dh ? 1 : 0) | (demb ? 2 : 0);
  const int cols = piece_columns(rows, vocab, piece);
  const HeadScratch at = head_scratch(rows, d, cols, grads);
  const size_t n = static_cast<size_t>(rows), table = static_cast<size_t>(vocab) * d;
  const Range in[4] = {{h, ((n - 1) * ldh + d) * 2},
                       {emb, table * 2},
                       {tokens + row0 + 1, (n - ((static_cast<int64_t>(row0) + rows) % seq == 0)) * 4},
                       {row_weight, row_weight ? n * 4 : 0}};
  const Range out[4] = {{loss_rows, n * 4},
                        {dh, dh ? ((n - 1) * lddh + d) * 2 : 0},
                        {demb, demb ? table * (demb_dtype == DT_F32 ? 4 : 2) : 0},
                        {scratch, at.bytes}};
  for (int i = 0; i < 4; ++i) {
    if (attn::overlaps(out[i], {in[0], in[1], in[2], in[3]}))
      return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: an output or the scratch overlaps an input");
    for (int j = 0; j < i; ++j)
      if (attn::overlaps(out[i], {out[j]}))
        return set_error(GPIPE_ERR_INVALID_ARG, "head_loss: outputs and scratch may not overlap each other");
  }
  int* err = device_error_ptr();
  if (!err) return set_error(GPIPE_ERR_CUDA, "head_loss: no device error word");

  char* w = static_cast<char*>(scratch);
  auto* info = reinterpret_cast<HeadRow*>(w + at.info);
  auto* hm = reinterpret_cast<__nv_bfloat16*>(w + at.hm);
  float* z = reinterpret_cast<float*>(w + at.z);
  auto* g = reinterpret_cast<__nv_bfloat16*>(w + at.g);
  float* dh32 = reinterpret_cast<float*>(w + at.dh);
  const HeadArgs a{rows, d, vocab, seq, row0, tokens, row_weight, inv_count, clip};
  int rc;
  (void)launch_k(head_rows_kernel, (rows + 7) / 8, 256, 0, st, a, static_cast<const __nv_bfloat16*>(h), ldh, hm, info,
                 err);
  if ((rc = check("rows"))) return rc;
  auto logits = [&](int v0, int kc) {
    GemmDesc q;
    q.M = rows;
    q.N = kc;
    q.K = d;
    q.A = hm;
    q.lda = d;
    q.B = static_cast<const __nv_bfloat16*>(emb) + static_cast<int64_t>(v0) * d;
    q.ldb = d;
    q.epi = EPI_STORE_F32;
    q.C = z;
    q.ldc = cols;
    return launch_gemm(q, st);
  };
  for (int v0 = 0; v0 < vocab; v0 += cols) {
    const int kc = std::min(cols, vocab - v0);
    if ((rc = logits(v0, kc))) return rc;
    (void)launch_k(head_stats_kernel, rows, 256, 0, st, a, static_cast<const float*>(z), static_cast<int64_t>(cols),
                   v0, kc, info);
    if ((rc = check("stats"))) return rc;
  }
  (void)launch_k(head_loss_kernel, (rows + 255) / 256, 256, 0, st, rows, inv_count, static_cast<const HeadRow*>(info),
                 loss_rows);
  if ((rc = check("loss"))) return rc;
  if (!grads) return GPIPE_OK;
  if (dh && cudaMemsetAsync(dh32, 0, n * d * 4, st) != cudaSuccess)
    return set_error(GPIPE_ERR_CUDA, "head_loss: memset");
  for (int v0 = 0; v0 < vocab; v0 += cols) {
    const int kc = std::min(cols, vocab - v0);
    if ((rc = logits(v0, kc))) return rc;
    (void)launch_k(head_grad_kernel, rows, 256, 0, st, a, static_cast<const float*>(z), static_cast<int64_t>(cols), v0,
                   kc, static_cast<const HeadRow*>(info), g);
    if ((rc = check("gradient"))) return rc;
    const int64_t row_of = static_cast<int64_t>(v0) * d;
    GemmDesc q;
    q.ldb = d;
    q.N = d;
    q.b_kmajor = false;
    q.A = g;
    q.lda = cols;
    q.ldc = d;
    if (dh) {
      q.M = rows;
      q.K = kc;
      q.B = static_cast<const __nv_bfloat16*>(emb) + row_of;
      q.epi = EPI_ACC_F32;
      q.C = dh32;
      if ((rc = launch_gemm(q, st))) return rc;
    }
    if (demb) {
      q.M = kc;
      q.K = rows;
      q.a_kmajor = false;
      q.B = hm;
      q.epi = demb_dtype == DT_F32 ? EPI_ACC_F32 : EPI_STORE;
      q.C = demb_dtype == DT_F32 ? static_cast<void*>(static_cast<float*>(demb) + row_of)
                                 : static_cast<void*>(static_cast<__nv_bfloat16*>(demb) + row_of);
      if ((rc = launch_gemm(q, st))) return rc;
    }
  }
  if (!dh) return GPIPE_OK;
  (void)launch_k(head_dh_kernel, (rows + 7) / 8, 256, 0, st, rows, d, static_cast<const float*>(dh32),
                 static_cast<__nv_bfloat16*>(dh), lddh);
  return check("dh");
}

}  // namespace gp
