// Distillation from a teacher's top logits, with the hard-label cross-entropy
// beside it, and the gradient of both in the same pass over the logits.
//
// Per row, with student logits z, teacher logits t_k at tokens idx_k (a slot
// with idx_k < 0 is empty), p = softmax(t / T) over the filled slots and
// q_T = softmax(z / T):
//   loss = kd T^2 sum_k p_k (log p_k - log q_T[idx_k]) + ce (-log q_1[target])
//   dz   = kd T (q_T - sum_k p_k onehot(idx_k)) + ce (q_1 - onehot(target))
// T^2 keeps the size of the gradient at any temperature.  A row without a
// filled slot has no teacher term, one without a target no label term.
//
// The operator is bound by memory: a row is read once and written once.
//
// Both softmaxes share the maximum m of z: q_T = e^{(z - m) / T} / s_T.  The
// subtraction comes first, so the exponent is exact to fp32 however large the
// logits are; so it does in p.  The top tokens are few, so dz is written as if there were none
// and their elements are written again; slots that name the same token are
// added by the first of them, in slot order, so that nothing depends on timing.
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "../../include/gpipe.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_util.cuh"

namespace gp {
namespace {

using attn::al16;
using attn::kLog2e;

constexpr int kDistillThreads = 512;
constexpr int kMaxTop = 256;

struct DistillArgs {
  int vocab, topk, seq, row0;
  int64_t ld, lddz;
  const int32_t* top_idx;
  const float* top_logit;
  const int32_t* tokens;
  float inv_t, kd, ce;  // 1 / T; kd T^2; ce
  float kd_grad;        // kd T
  float* loss;
  int* err;
  bool in_place;
};

// V consecutive elements as floats: 16 bytes a load, or one element.
template <typename T, bool VEC>
struct Vec {
  static constexpr int N = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  static __device__ __forceinline__ void load(const T* p, float* v) {
    if constexpr (!VEC) {
      v[0] = Elem<T>::ld(p);
    } else if constexpr (sizeof(T) == 2) {
      load8(p, v);
    } else {
      const float4 x = *reinterpret_cast<const float4*>(p);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    if constexpr (!VEC) {
      *p = f2bf(v[0]);
    } else if constexpr (N == 8) {
      store8(p, v);
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  }
};

__device__ __forceinline__ void join(float& m, float& s, float& st, float om, float os, float ost, float c1, float ct) {
  const float nm = fmaxf(m, om);
  // a side that saw nothing has sums 0 and maximum -inf
  const float a = m == -INFINITY ? m : m - nm, b = om == -INFINITY ? om : om - nm;
  s = s * ex2_approx(a * c1) + os * ex2_approx(b * c1);
  st = st * ex2_approx(a * ct) + ost * ex2_approx(b * ct);
  m = nm;
}

// The teacher's side of a row, by one warp: p over the filled slots into pk (all
// zero without one) and log p in place of the logits tl.  Returns whether any slot
// is filled.
__device__ __forceinline__ bool teacher(const DistillArgs& a, float* tl, float* pk, int lane) {
  float tm = -INFINITY;
  for (int k = lane; k < a.topk; k += 32) tm = fmaxf(tm, tl[k]);
  tm = warp_max(tm);
  const float tb = tm == -INFINITY ? 0.f : tm;
  float ts = 0.f;
  for (int k = lane; k < a.topk; k += 32) {
    tl[k] = (tl[k] - tb) * a.inv_t;
    ts += pk[k] = expf(tl[k]);
  }
  ts = warp_sum(ts);
  const float log_ts = logf(ts);
  for (int k = lane; k < a.topk; k += 32) {
    pk[k] = ts == 0.f ? 0.f : pk[k] / ts;
    tl[k] -= log_ts;
  }
  return ts != 0.f;
}
// sum p (log p - log q_T), by one warp.
__device__ __forceinline__ float divergence(const DistillArgs& a, const float* lp, const float* zt, const float* pk,
                                            float m, float st, int lane) {
  const float log_st = logf(st);
  float x = 0.f;
  for (int k = lane; k < a.topk; k += 32)
    if (pk[k] != 0.f) x += pk[k] * (lp[k] - ((zt[k] - m) * a.inv_t - log_st));
  return warp_sum(x);
}

// The target of row r, or -1; an id outside the vocabulary is flagged (by `flag`).
__device__ __forceinline__ int target_of(const DistillArgs& a, int64_t r, bool flag) {
  if (!(a.ce > 0.f)) return -1;
  const int64_t g = a.row0 + r;
  if (g % a.seq == a.seq - 1) return -1;
  const int t = a.tokens[g + 1];
  if (t >= 0 && t < a.vocab) return t;
  if (flag) atomicExch(a.err, DERR_BAD_TOKEN);
  return -1;
}

// Write the element of slot or target `me` (student logit x + m), once: by the
// first slot that names it, or the target's thread (k = topk) if none does.
__device__ __forceinline__ void fix_up(const DistillArgs& a, const int* idx, const float* pk, int k, int me, float x,
                                       int target, float gt, float g1, __nv_bfloat16* out) {
  float p = 0.f;
  bool first = true;
  for (int i = 0; i < a.topk; ++i)
    if (idx[i] == me) {
      if (i < k) first = false;
      p += pk[i];
    }
  if (!first) return;
  float g = gt != 0.f ? ex2_approx(x * (kLog2e * a.inv_t)) * gt - a.kd_grad * p : 0.f;
  if (g1 != 0.f) g += ex2_approx(x * kLog2e) * g1;
  if (me == target) g -= a.ce;
  out[me] = f2bf(g);
}

// ---------------------------------------------------------------------------
// A row in registers
// ---------------------------------------------------------------------------
// A CTA takes a row, 16 bytes a load (one element, where rows do not start on
// 16-byte boundaries) and up to NV loads a thread, all of them issued before the
// first is used.  The row is read once and dz is made from the registers: the bytes
// the operator cannot do without and no others.  The teacher's side is made while the row's loads are on their way.
// Short rows take CTAs of 64 threads, so that many of them are under way on an
// SM: a row's time is a chain of loads, sums and stores however short it is.
//
// What a thread keeps of its row: NV vectors as they came.
template <typename T, bool VEC, int NV, int TH>
struct Slice {
  static constexpr int E = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  static constexpr int kElems = TH * NV * E;
  using Word = typename std::conditional<VEC, uint4, float>::type;
  Word w[NV];

  __device__ __forceinline__ void load(const T* z, int n, int tid) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = (j * TH + tid) * E;
      if constexpr (VEC) {
        if (i + E <= n) {
          w[j] = *reinterpret_cast<const uint4*>(z + i);
        } else if constexpr (sizeof(T) == 4) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = i + e < n ? z[i + e] : -INFINITY;
          w[j] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        } else {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = i + e < n ? Elem<T>::ld(z + i + e) : -INFINITY;
          w[j] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                            pack_bf16x2(v[6], v[7]));
        }
      } else {
        w[j] = i < n ? Elem<T>::ld(z + i) : -INFINITY;
      }
    }
  }
  __device__ __forceinline__ void get(int j, float* v) const {
    if constexpr (!VEC) {
      v[0] = w[j];
    } else if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(w[j].x);
      v[1] = __uint_as_float(w[j].y);
      v[2] = __uint_as_float(w[j].z);
      v[3] = __uint_as_float(w[j].w);
    } else {
      const float2 a = unpack_bf16x2(w[j].x), b = unpack_bf16x2(w[j].y), c = unpack_bf16x2(w[j].z),
                   d = unpack_bf16x2(w[j].w);
      v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y; v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
    }
  }
};

template <typename T, bool VEC, int NV, int TH>
__global__ void __launch_bounds__(TH) distill_row_kernel(const T* logits, __nv_bfloat16* dz,
                                                         const __grid_constant__ DistillArgs a) {
  griddep_wait();
  griddep_launch();
  using S = Slice<T, VEC, NV, TH>;
  constexpr int E = S::E, W = TH / 32;
  __shared__ float sm_m[W], sm_s[W], sm_t[W];
  __shared__ int idx[kMaxTop];
  __shared__ float tl[kMaxTop], zt[kMaxTop], pk[kMaxTop];
  __shared__ float sh_z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t r = blockIdx.x;
  const int n = a.vocab;
  const T* z = logits + r * a.ld;
  const float c1 = kLog2e, ct = kLog2e * a.inv_t;

  S row;
  row.load(z, n, tid);
  const int target = target_of(a, r, tid == 0);
  for (int k = tid; k < a.topk; k += TH) {
    int i = a.top_idx[r * a.topk + k];
    if (i >= a.vocab) {
      atomicExch(a.err, DERR_BAD_TOKEN);
      i = -1;
    }
    idx[k] = i;
    tl[k] = i >= 0 ? a.top_logit[r * a.topk + k] : -INFINITY;
    zt[k] = i >= 0 ? Elem<T>::ld(z + i) : 0.f;
  }
  if (tid == 0 && target >= 0) sh_z = Elem<T>::ld(z + target);
  __syncthreads();
  __shared__ float sh_has;
  if (warp == W - 1) {
    const bool has = teacher(a, tl, pk, lane);
    if (lane == 0) sh_has = has ? 1.f : 0.f;
  }

  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[E];
    row.get(j, v);
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, v[e]);
  }
  float s1 = 0.f, st = 0.f;
  {
    const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[E];
      row.get(j, v);
      if (E * j * TH < n) {  // (uniform)
#pragma unroll
        for (int e = 0; e < E; ++e) st += ex2_approx((v[e] - ms) * ct);
        if (a.ce > 0.f) {
#pragma unroll
          for (int e = 0; e < E; ++e) s1 += ex2_approx((v[e] - ms) * c1);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s1, o),
                ot = __shfl_xor_sync(0xffffffffu, st, o);
    join(m, s1, st, om, os, ot, c1, ct);
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_s[warp] = s1;
    sm_t[warp] = st;
  }
  __syncthreads();
  m = sm_m[0];
  s1 = sm_s[0];
  st = sm_t[0];
#pragma unroll
  for (int w = 1; w < W; ++w) join(m, s1, st, sm_m[w], sm_s[w], sm_t[w], c1, ct);
  if (warp == W - 1) {
    const float kl = divergence(a, tl, zt, pk, m, st, lane);
    if (lane == 0) {
      float loss = a.kd * kl;
      if (target >= 0) loss += a.ce * (logf(s1) - (sh_z - m));
      a.loss[r] = loss;
    }
  }
  if (dz) {
    const float gt = sh_has != 0.f ? a.kd_grad / st : 0.f;
    const float g1 = target >= 0 ? a.ce / s1 : 0.f;
    __nv_bfloat16* out = dz + r * a.lddz;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = (j * TH + tid) * E;
      if (i < n) {
        float v[E], g[E];
        row.get(j, v);
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = gt != 0.f ? ex2_approx((v[e] - m) * ct) * gt : 0.f;
        if (g1 != 0.f) {
#pragma unroll
          for (int e = 0; e < E; ++e) g[e] = fmaf(ex2_approx((v[e] - m) * c1), g1, g[e]);
        }
        if (i + E <= n) {
          Vec<T, VEC>::store(out + i, g);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (i + e < n) out[i + e] = f2bf(g[e]);
        }
      }
    }
    __syncthreads();
    // the elements of the top tokens and of the target, once each
    for (int k = tid; k < a.topk; k += TH) {
      const int me = idx[k];
      if (me >= 0) fix_up(a, idx, pk, k, me, zt[k] - m, target, gt, g1, out);
    }
    if (tid == 0 && target >= 0) fix_up(a, idx, pk, a.topk, target, sh_z - m, target, gt, g1, out);
  }
}

// ---------------------------------------------------------------------------
// Rows in a stream
// ---------------------------------------------------------------------------
// A cluster of C CTAs, one on an SM, takes rows one after the other, each CTA a
// slice of them.  Slices pass through a ring of 32 KB chunks in shared memory:
// the copies run ahead by whatever the ring has left beside the current slice,
// so that memory is never idle while a row's sums are joined, and a row is read
// from memory once although it is used twice.
//   warp 20      copies: the chunks of row after row, as the ring empties.
//   warps 0-15   pass A over a slice's chunks (maximum and sums), joined over the
//                warps and, through remote shared memory, over the cluster; pass
//                B over the same chunks, which writes dz and frees them.  For the loss alone
//                pass A frees them, and a slice may be longer than the ring.
//   warps 16-19  two groups, of the even and the odd rows: the teacher of a row ahead
//                of time (its tokens, the student's logits there, p), then, once its
//                sums are known, its loss and, once pass B is done, the elements of
//                its top tokens.
//
// Bound by memory where the label term is off (4096 x 131072 bf16: 372 us, 5.8
// TB/s); with it, four exponentials and some 14 instructions an element share the
// bound with it (2048 x 32000 fp32: 77 us, 5.2 TB/s, an SM's quarters issuing in
// 64 % of the cycles; 4096 x 131072 bf16: 474 us).  Part of the label's
// exponentials as polynomials, for the exponentials' unit's sake, made 511 us of 473
// (a quarter of them) and 667 us (all).  One CTA of 512 pass threads was as fast
// as two of half the ring, and 64 teacher threads a group leave the pass warps the
// registers that 128 do not (381 and 395 us).
constexpr int kChunk = 32768, kChunks = 6, kMaxSliceChunks = 4;
constexpr int kPassThreads = 512, kTeachThreads = 64, kStreamThreads = kPassThreads + 2 * kTeachThreads + 32;
constexpr int kSlots = kMaxTop / kTeachThreads;  // slots a teacher thread
constexpr int kMaxCluster = 8;

struct StreamShared {
  uint64_t full[kChunks], empty[kChunks];
  uint64_t ready[2];  // the teacher of a row of this parity is known (kTeachThreads arrivals)
  uint64_t sums[2];   // its maximum and sums are
  uint64_t done[2];   // its pass B is (one arrival a warp)
  uint64_t cross[2];  // every CTA of the cluster has sent its sums
  float part[2][3][kPassThreads / 32];
  float sent[2][kMaxCluster][4];
  float total[2][4];
  float has[2], label[2];  // whether the row has a teacher, a target
  __align__(16) int idx[2][kMaxTop];
  float pk[2][kMaxTop];
  float kl[2][kTeachThreads / 32];
  int abort;
};
constexpr int kStreamSmem = kChunks * kChunk + static_cast<int>(sizeof(StreamShared));

__device__ __forceinline__ void pass_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kPassThreads) : "memory"); }
__device__ __forceinline__ void teach_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(2 + group), "n"(kTeachThreads) : "memory");
}

// What a teacher thread has of its slots of a row, step by step.
struct Fetched {
  int id[kSlots];
  float logit[kSlots];
  int target;
};
struct Gathered {
  int id[kSlots];
  float tl[kSlots], z[kSlots];
  int target;
  float zt;
};
struct Slots {
  int me[kSlots];   // the token, or -1 (empty, or named by an earlier slot)
  float z[kSlots];  // the student's logit there
  float p[kSlots];  // the slot's probability, and log p
  float logp[kSlots];
  float sum[kSlots];  // over all slots of that token
  int target;
  float zt;
  bool fix_target;  // the target's element is this thread's: no slot names it
};

// GRAD: the loss alone, or with dz by wide stores, or, where a row of dz is not aligned
// for them when its logits are, by single ones (2048 x 32001 logits in rows of 32008, dz
// in rows of 32001, bf16: 91 us; 81 where both are alike, 150 with rows read twice).
// ROWS: any, or those that all start on a 16-byte boundary, so that a CTA's part is the
// same of all rows and made once, or those that also end on one, so that nothing is read
// beside the copies.  4096 x 131072 bf16 372 us, 381 as rows that may end anywhere; with
// labels 474, 492 with a part made row by row.
enum Grad { kLoss, kWide, kSingle };
enum Rows { kAny, kAligned, kWhole };
template <typename T, bool CE, Grad GRAD, Rows ROWS>
__global__ void __launch_bounds__(kStreamThreads, 1)
    distill_stream_kernel(const T* logits, __nv_bfloat16* dz, const __grid_constant__ DistillArgs a, int rows, int ctas,
                          int per) {
  extern __shared__ __align__(128) uint8_t ring[];
  StreamShared& sh = *reinterpret_cast<StreamShared*>(ring + kChunks * kChunk);
  volatile int* abort = &sh.abort;
  constexpr bool ALIGNED = ROWS != kAny, EDGES = ROWS != kWhole;
  constexpr int E = 16 / static_cast<int>(sizeof(T)), kPer = kChunk / static_cast<int>(sizeof(T));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % ctas, clusters = gridDim.x / ctas;
  // This CTA's part of row r: elements lo .. hi - 1, of which `whole` from the first
  // 16-byte boundary on come by copies and the few before and behind them are read directly.
  struct Part {
    int lo, hi, from, whole, chunks;
  };
  auto part_of = [&](int64_t r) {
    // (in 32 bits: E is a power of two, and only the low bits count)
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(logits) / sizeof(T)) +
                        static_cast<uint32_t>(r) * static_cast<uint32_t>(a.ld);
    Part p;
    p.from = (ALIGNED ? 0 : static_cast<int>(-at & (E - 1))) + rank * per;
    p.lo = rank ? min(p.from, a.vocab) : 0;
    p.hi = min(a.vocab, p.from + per);
    p.whole = max(0, p.hi - p.from) / E * E;
    p.chunks = (p.whole + kPer - 1) / kPer;
    return p;
  };
  const int row0 = blockIdx.x / ctas;
  const Part fixed = part_of(0);  // of every row, where ALIGNED
  const float c1 = kLog2e, ct = kLog2e * a.inv_t;

  if (tid == 0) {
    for (int i = 0; i < kChunks; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kPassThreads / 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.ready[i], kTeachThreads);
      mbar_init(&sh.sums[i], 1);
      mbar_init(&sh.done[i], kPassThreads / 32);
      mbar_init(&sh.cross[i], ctas);
    }
    sh.abort = 0;
    fence_barrier_init();
  }
  griddep_wait();
  if (ctas > 1) cluster_sync();  // the peers' barriers are there before anything is sent to them
  else __syncthreads();

  if (warp == kStreamThreads / 32 - 1) {  // ---- copies ----
    if (lane == 0) {
      int slot = 0;
      uint32_t parity = 1;  // of the wait for an empty slot; in the first round there is none
      int64_t count = 0;
      bool go = true;
      for (int r = row0; r < rows && go; r += clusters) {
        const Part p = ALIGNED ? fixed : part_of(r);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(logits + static_cast<int64_t>(r) * a.ld + p.from);
        for (int c = 0; c < p.chunks; ++c) {
          if (count >= kChunks && !lane_await(&sh.empty[slot], parity, a.err, DERR_TMA_WAIT, abort)) {
            go = false;
            break;
          }
          const uint32_t bytes = static_cast<uint32_t>(min(kPer, p.whole - c * kPer)) * sizeof(T);
          mbar_arrive_expect_tx(&sh.full[slot], bytes);
          bulk_load(ring + slot * kChunk, src + static_cast<int64_t>(c) * kChunk, bytes, &sh.full[slot]);
          ++count;
          if (++slot == kChunks) {
            slot = 0;
            parity ^= 1u;
          }
        }
      }
      // no copy may still be landing when the CTA exits
      for (int64_t k = count > kChunks ? count - kChunks : 0; k < count; ++k)
        mbar_wait_bounded(&sh.full[k % kChunks], static_cast<uint32_t>(k / kChunks) & 1u, a.err, DERR_DRAIN_WAIT);
    }
    __syncwarp();
  } else if (warp >= kPassThreads / 32) {  // ---- the teacher ----
    const int b = (tid - kPassThreads) / kTeachThreads;  // the group, and the parity of its rows
    const int t = tid - kPassThreads - b * kTeachThreads, w = t >> 5;
    // A row's tokens are loaded two of this group's rows ahead, the student's logits
    // there one ahead, before the row in hand is finished.
    auto fetch = [&](int64_t r) {
      Fetched f;
      f.target = -1;
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        f.id[k] = -1;
        f.logit[k] = 0.f;
      }
      if (r >= rows) return f;
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        const int slot = t + k * kTeachThreads;
        if (slot < a.topk) {
          f.id[k] = a.top_idx[r * a.topk + slot];
          f.logit[k] = a.top_logit[r * a.topk + slot];
        }
      }
      f.target = target_of(a, r, rank == 0 && t == 0);
      return f;
    };
    auto gather = [&](const Fetched& f, int64_t r) {
      Gathered g;
      const T* z = logits + r * a.ld;
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        int i = f.id[k];
        if (i >= a.vocab) {
          if (rank == 0) atomicExch(a.err, DERR_BAD_TOKEN);
          i = -1;
        }
        g.id[k] = i;
        g.tl[k] = i >= 0 ? f.logit[k] : -INFINITY;
        g.z[k] = i >= 0 ? Elem<T>::ld(z + i) : 0.f;
      }
      g.target = f.target;
      g.zt = f.target >= 0 ? Elem<T>::ld(z + f.target) : 0.f;
      return g;
    };
    auto prepare = [&](const Gathered& g) {
      Slots s;
      s.target = g.target;
      s.zt = g.zt;
      const int* id = g.id;
      const float* tl = g.tl;
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        const int slot = t + k * kTeachThreads;
        s.z[k] = g.z[k];
        sh.idx[b][slot] = id[k];  // (-1 behind the last slot too)
        sh.pk[b][slot] = tl[k];
      }
      teach_sync(b);
      // every warp takes the maximum and the sum over all slots by itself
      float tm = -INFINITY;
      for (int k = lane; k < a.topk; k += 32) tm = fmaxf(tm, sh.pk[b][k]);
      tm = warp_max(tm);
      const float tb = tm == -INFINITY ? 0.f : tm;
      float ts = 0.f;
      for (int k = lane; k < a.topk; k += 32) ts += expf((sh.pk[b][k] - tb) * a.inv_t);
      ts = warp_sum(ts);
      const float log_ts = logf(ts);
      teach_sync(b);
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        const int slot = t + k * kTeachThreads;
        const float x = (tl[k] - tb) * a.inv_t;
        s.p[k] = ts == 0.f || id[k] < 0 ? 0.f : expf(x) / ts;
        s.logp[k] = x - log_ts;
        sh.pk[b][slot] = s.p[k];
      }
      if (t == 0) {
        sh.has[b] = ts == 0.f ? 0.f : 1.f;
        sh.label[b] = s.target >= 0 ? 1.f : 0.f;
      }
      teach_sync(b);
      // slots of the same token: usually there are none but the slot itself
      s.fix_target = t == 0 && s.target >= 0;
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        s.me[k] = id[k];
        s.sum[k] = 0.f;
      }
      const int4* all = reinterpret_cast<const int4*>(sh.idx[b]);
      for (int i = 0; i < (a.topk + 3) / 4; ++i) {
        const int4 v = all[i];
        const int four[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
          if (id[k] >= 0 && (v.x == id[k] || v.y == id[k] || v.z == id[k] || v.w == id[k])) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (four[j] == id[k]) {
                if (4 * i + j < t + k * kTeachThreads) s.me[k] = -1;
                s.sum[k] += sh.pk[b][4 * i + j];
              }
          }
        if (s.fix_target && (v.x == s.target || v.y == s.target || v.z == s.target || v.w == s.target))
          s.fix_target = false;
      }
      mbar_arrive1(&sh.ready[b]);
      return s;
    };
    auto finish = [&](const Slots& s, int r, uint32_t parity) {
      (void)lane_await(&sh.sums[b], parity, a.err, DERR_ACC_WAIT, abort);
      __syncwarp();
      const float m = sh.total[b][0], s1 = sh.total[b][1], st = sh.total[b][2];
      if (rank == 0) {
        const float log_st = logf(st);
        float kl = 0.f;
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
          if (s.p[k] != 0.f) kl += s.p[k] * (s.logp[k] - ((s.z[k] - m) * a.inv_t - log_st));
        kl = warp_sum(kl);
        if (lane == 0) sh.kl[b][w] = kl;
        teach_sync(b);
        if (t == 0) {
          float loss = 0.f;
          for (int i = 0; i < kTeachThreads / 32; ++i) loss += sh.kl[b][i];
          loss *= a.kd;
          if (s.target >= 0) loss += a.ce * (logf(s1) - (s.zt - m));
          a.loss[r] = loss;
        }
      }
      // (without dz too: a pass warp must have seen this row's teacher before the next one's is ready)
      (void)lane_await(&sh.done[b], parity, a.err, DERR_ACC_WAIT, abort);
      __syncwarp();
      if (GRAD == kLoss) return;
      const float gt = sh.has[b] != 0.f ? a.kd_grad / st : 0.f;
      const float g1 = s.target >= 0 ? a.ce / s1 : 0.f;
      __nv_bfloat16* out = dz + static_cast<int64_t>(r) * a.lddz;
      auto value = [&](float x, float p, bool is_target) {
        float g = gt != 0.f ? ex2_approx(x * ct) * gt - a.kd_grad * p : 0.f;
        if (g1 != 0.f) g += ex2_approx(x * c1) * g1;
        return f2bf(is_target ? g - a.ce : g);
      };
      const Part part = ALIGNED ? fixed : part_of(r);
#pragma unroll
      for (int k = 0; k < kSlots; ++k)
        if (s.me[k] >= part.lo && s.me[k] < part.hi) out[s.me[k]] = value(s.z[k] - m, s.sum[k], s.me[k] == s.target);
      if (s.fix_target && s.target >= part.lo && s.target < part.hi) out[s.target] = value(s.zt - m, 0.f, true);
    };
    const int64_t first = row0 + static_cast<int64_t>(b) * clusters, stride = 2 * static_cast<int64_t>(clusters);
    Gathered g = {};
    if (first < rows) g = gather(fetch(first), first);
    Fetched f = fetch(first + stride);
    uint32_t parity = 0;
    for (int64_t r = first; r < rows; r += stride, parity ^= 1u) {
      const Slots cur = prepare(g);
      if (r + stride < rows) g = gather(f, r + stride);
      f = fetch(r + 2 * stride);
      finish(cur, static_cast<int>(r), parity);
    }
  } else {  // ---- passes ----
    constexpr int V = kPer / (E * kPassThreads);  // vectors a thread takes of a chunk
    const f32x2 c12 = pack2(c1, c1), ct2 = pack2(ct, ct);
    auto load_chunk = [&](const T* at, int left, float* v) {  // elements behind the `left` of a last chunk: -inf
      at += tid * E;
#pragma unroll
      for (int j = 0; j < V; ++j) Vec<T, true>::load(at + j * kPassThreads * E, v + j * E);
      if (left < kPer) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if ((j * kPassThreads + tid) * E >= left) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[j * E + e] = -INFINITY;
          }
      }
    };
    int slot = 0, i = 0;
    uint32_t parity = 0;
    for (int r = row0; r < rows; r += clusters, ++i) {
      const int b = i & 1;
      const uint32_t turn = (i >> 1) & 1;
      const Part p = ALIGNED ? fixed : part_of(r);
      const int whole = p.whole, chunks = p.chunks;
      // the first and the last few elements, one a thread, kept for pass B (dz may lie over them by then)
      auto edge_of = [&] {
        if (!EDGES) return -1;
        if (ALIGNED) return p.from + whole + tid < p.hi ? p.from + whole + tid : -1;
        const int at = tid < 16 ? tid : p.from + whole + tid - 16;
        return tid < 32 && at >= p.lo && at < (tid < 16 ? p.from : p.hi) ? at : -1;
      };
      float edge = -INFINITY;
      const int at_edge = edge_of();
      if (EDGES && at_edge >= 0) edge = Elem<T>::ld(logits + static_cast<int64_t>(r) * a.ld + at_edge);
      // pass A: running maximum (one check a chunk) and the sums
      float m = edge;
      f32x2 s12 = 0ull, st2 = 0ull;
      if (EDGES && at_edge >= 0) s12 = st2 = pack2(edge == -INFINITY ? 0.f : ex2_approx(edge - edge), 0.f);  // 1 (NaN stays NaN)
      int sl = slot;
      uint32_t pa = parity;
      for (int c = 0; c < chunks; ++c) {
        (void)lane_await(&sh.full[sl], pa, a.err, DERR_ACC_WAIT, abort);
        __syncwarp();
        float v[V * E];
        load_chunk(reinterpret_cast<const T*>(ring + sl * kChunk), min(kPer, whole - c * kPer), v);
        float mx = v[0];
#pragma unroll
        for (int e = 1; e + 1 < V * E; e += 2) mx = fmax3(mx, v[e], v[e + 1]);
        mx = fmaxf(mx, v[V * E - 1]);
        if (mx > m) {
          const float d = m == -INFINITY ? m : m - mx;
          const float a1 = ex2_approx(d * c1), at = ex2_approx(d * ct);
          if (CE) s12 = mul2(s12, pack2(a1, a1));
          st2 = mul2(st2, pack2(at, at));
          m = mx;
        }
        const float ms = m == -INFINITY ? 0.f : -m;
        const f32x2 ms2 = pack2(ms, ms);
#pragma unroll
        for (int e = 0; e < V * E; e += 2) {
          const f32x2 d = add2(pack2(v[e], v[e + 1]), ms2);
          float x0, x1;
          unpack2(mul2(d, ct2), x0, x1);
          st2 = add2(st2, pack2(ex2_approx(x0), ex2_approx(x1)));
          if (CE) {
            unpack2(mul2(d, c12), x0, x1);
            s12 = add2(s12, pack2(ex2_approx(x0), ex2_approx(x1)));
          }
        }
        if (GRAD == kLoss) {  // no pass B
          __syncwarp();
          if (lane == 0) mbar_arrive1(&sh.empty[sl]);
        }
        if (++sl == kChunks) {
          sl = 0;
          pa ^= 1u;
        }
      }
      float s1, st, half;
      unpack2(s12, s1, half);
      s1 += half;
      unpack2(st2, st, half);
      st += half;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s1, o),
                    ot = __shfl_xor_sync(0xffffffffu, st, o);
        join(m, s1, st, om, os, ot, c1, ct);
      }
      if (lane == 0) {
        sh.part[b][0][warp] = m;
        sh.part[b][1][warp] = s1;
        sh.part[b][2][warp] = st;
      }
      pass_sync();
      {  // every warp joins the warps' sums by itself
        constexpr int W = kPassThreads / 32;
        m = lane < W ? sh.part[b][0][lane] : -INFINITY;
        s1 = lane < W ? sh.part[b][1][lane] : 0.f;
        st = lane < W ? sh.part[b][2][lane] : 0.f;
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) {
          const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s1, o),
                      ot = __shfl_xor_sync(0xffffffffu, st, o);
          join(m, s1, st, om, os, ot, c1, ct);
        }
        m = __shfl_sync(0xffffffffu, m, 0);
        s1 = __shfl_sync(0xffffffffu, s1, 0);
        st = __shfl_sync(0xffffffffu, st, 0);
      }
      // the teacher has read the logits of this row that it needs: dz may be written over them
      (void)lane_await(&sh.ready[b], turn, a.err, DERR_ACC_WAIT, abort);
      __syncwarp();
      if (ctas > 1) {
        if (tid < ctas) {  // to every CTA, this one among them
          const uint32_t at = map_peer(smem_u32(sh.sent[b][rank]), lane);
          st_peer_f32(at, m);
          st_peer_f32(at + 4, s1);
          st_peer_f32(at + 8, st);
          mbar_arrive_cluster(map_peer(smem_u32(&sh.cross[b]), lane));
        }
        (void)lane_await_cluster(&sh.cross[b], turn, a.err, DERR_ACC_WAIT, abort);
        __syncwarp();
        m = -INFINITY;
        s1 = st = 0.f;
        for (int c = 0; c < ctas; ++c)  // in rank order, the same in every CTA
          join(m, s1, st, sh.sent[b][c][0], sh.sent[b][c][1], sh.sent[b][c][2], c1, ct);
      }
      if (tid == 0) {
        sh.total[b][0] = m;
        sh.total[b][1] = s1;
        sh.total[b][2] = st;
        mbar_arrive1(&sh.sums[b]);
      }
      if (GRAD == kLoss) {
        slot = sl;
        parity = pa;
        __syncwarp();
        if (lane == 0) mbar_arrive1(&sh.done[b]);
        continue;
      }
      // pass B
      const float gt = sh.has[b] != 0.f ? a.kd_grad / st : 0.f;
      const float g1 = sh.label[b] != 0.f ? a.ce / s1 : 0.f;
      __nv_bfloat16* out = dz + static_cast<int64_t>(r) * a.lddz + p.from;
      const f32x2 m2 = pack2(-m, -m), gt2 = pack2(gt, gt), g12 = pack2(g1, g1);
      // dz of pairs, by which of the two terms the row has
      auto pass_b = [&](auto grad2) {
        for (int c = 0; c < chunks; ++c) {
          const int left = min(kPer, whole - c * kPer);
          const T* chunk = reinterpret_cast<const T*>(ring + slot * kChunk);
          float v[V * E];
          if constexpr (GRAD == kWide) {
            load_chunk(chunk, left, v);
          } else {  // element by element, neighbours to neighbouring threads
#pragma unroll
            for (int e = 0; e < V * E; ++e) {
              const int at = e * kPassThreads + tid;
              v[e] = at < left ? Elem<T>::ld(chunk + at) : -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < V * E; e += 2) unpack2(grad2(add2(pack2(v[e], v[e + 1]), m2)), v[e], v[e + 1]);
          __nv_bfloat16* to = out + c * kPer;
          if constexpr (GRAD == kWide) {
            to += tid * E;
            if (left == kPer) {
#pragma unroll
              for (int j = 0; j < V; ++j) Vec<T, true>::store(to + j * kPassThreads * E, v + j * E);
            } else {
#pragma unroll
              for (int j = 0; j < V; ++j)
                if ((j * kPassThreads + tid) * E < left) Vec<T, true>::store(to + j * kPassThreads * E, v + j * E);
            }
          } else {
#pragma unroll
            for (int e = 0; e < V * E; ++e) {
              const int at = e * kPassThreads + tid;
              if (at < left) to[at] = f2bf(v[e]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive1(&sh.empty[slot]);
          if (++slot == kChunks) {
            slot = 0;
            parity ^= 1u;
          }
        }
        if (EDGES && at_edge >= 0) {
          float g, other;
          unpack2(grad2(add2(pack2(edge, edge), m2)), g, other);
          out[at_edge - p.from] = f2bf(g);
        }
      };
      auto exps = [&](f32x2 d, f32x2 scale) {
        float x0, x1;
        unpack2(mul2(d, scale), x0, x1);
        return pack2(ex2_approx(x0), ex2_approx(x1));
      };
      if (gt != 0.f && (!CE || g1 == 0.f))
        pass_b([&](f32x2 d) { return mul2(exps(d, ct2), gt2); });
      else if (CE && gt != 0.f)
        pass_b([&](f32x2 d) { return fma2(exps(d, c12), g12, mul2(exps(d, ct2), gt2)); });
      else if (CE && g1 != 0.f)
        pass_b([&](f32x2 d) { return mul2(exps(d, c12), g12); });
      else
        pass_b([&](f32x2) { return f32x2(0); });
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sh.done[b]);
    }
  }
  // the peers may still be sending to this CTA
  if (ctas > 1) cluster_sync();
}

// ---------------------------------------------------------------------------
// A row in two passes
// ---------------------------------------------------------------------------
// For rows that no cluster holds, and for short unaligned ones, which the second pass
// still finds in L2 (figures at launch_rows).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kDistillThreads) distill_kernel(const T* logits,
                                                                 __nv_bfloat16* dz, DistillArgs a) {
  griddep_wait();
  griddep_launch();
  using V = Vec<T, VEC>;
  constexpr int W = kDistillThreads / 32;
  __shared__ float sm_m[W], sm_s[W], sm_t[W];
  __shared__ float sh[3];  // m, sum at 1, sum at T
  __shared__ int idx[kMaxTop];
  __shared__ float tl[kMaxTop], zt[kMaxTop], pk[kMaxTop];
  __shared__ float sh_z, sh_has;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const T* z = logits + r * a.ld;
  const float c1 = kLog2e, ct = kLog2e * a.inv_t;

  const int target = target_of(a, r, tid == 0);
  if (tid < a.topk) {
    int i = a.top_idx[r * a.topk + tid];
    if (i >= a.vocab) {
      atomicExch(a.err, DERR_BAD_TOKEN);
      i = -1;
    }
    idx[tid] = i;
    tl[tid] = i >= 0 ? a.top_logit[r * a.topk + tid] : -INFINITY;
    zt[tid] = i >= 0 ? Elem<T>::ld(z + i) : 0.f;
  }
  if (tid == 0 && target >= 0) sh_z = Elem<T>::ld(z + target);

  // pass 1: running maximum and the sums of both softmaxes
  float m = -INFINITY, s1 = 0.f, st = 0.f;
  for (int i = tid * V::N; i < a.vocab; i += kDistillThreads * V::N) {
    float v[V::N];
    if (i + V::N <= a.vocab) {
      V::load(z + i, v);
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e) v[e] = i + e < a.vocab ? Elem<T>::ld(z + i + e) : -INFINITY;
    }
    float mx = v[0];
#pragma unroll
    for (int e = 1; e < V::N; ++e) mx = fmaxf(mx, v[e]);
    if (mx > m) {
      const float d = m == -INFINITY ? m : m - mx;
      s1 *= ex2_approx(d * c1);
      st *= ex2_approx(d * ct);
      m = mx;
    }
    const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int e = 0; e < V::N; ++e) {
      if (a.ce > 0.f) s1 += ex2_approx((v[e] - ms) * c1);
      st += ex2_approx((v[e] - ms) * ct);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s1, o),
                ot = __shfl_xor_sync(0xffffffffu, st, o);
    join(m, s1, st, om, os, ot, c1, ct);
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_s[warp] = s1;
    sm_t[warp] = st;
  }
  __syncthreads();
  if (warp == 0) {
    m = lane < W ? sm_m[lane] : -INFINITY;
    s1 = lane < W ? sm_s[lane] : 0.f;
    st = lane < W ? sm_t[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s1, o),
                  ot = __shfl_xor_sync(0xffffffffu, st, o);
      join(m, s1, st, om, os, ot, c1, ct);
    }
    const bool has = teacher(a, tl, pk, lane);
    const float kl = divergence(a, tl, zt, pk, m, st, lane);
    if (lane == 0) {
      sh[0] = m;
      sh[1] = s1;
      sh[2] = st;
      sh_has = has ? 1.f : 0.f;
      float loss = a.kd * kl;
      if (target >= 0) loss += a.ce * (logf(s1) - (sh_z - m));
      a.loss[r] = loss;
    }
  }
  if (!dz) return;
  __syncthreads();
  m = sh[0];
  const float gt = sh_has != 0.f ? a.kd_grad / sh[2] : 0.f;
  const float g1 = target >= 0 ? a.ce / sh[1] : 0.f;
  __nv_bfloat16* out = dz + r * a.lddz;
  // pass 2.  In place, chunk c's elements are read by every thread before any is
  // written, and bf16 element i lies at or before the bytes of element i.
  for (int base = 0; base < a.vocab; base += kDistillThreads * V::N) {
    const int i = base + tid * V::N;
    float v[V::N];
    if (i + V::N <= a.vocab) {
      V::load(z + i, v);
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e) v[e] = i + e < a.vocab ? Elem<T>::ld(z + i + e) : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < V::N; ++e) {
      const float d = v[e] - m;
      float g = gt != 0.f ? ex2_approx(d * ct) * gt : 0.f;
      if (g1 != 0.f) g = fmaf(ex2_approx(d * c1), g1, g);
      v[e] = g;
    }
    if (a.in_place) __syncthreads();
    if (i + V::N <= a.vocab) {
      V::store(out + i, v);
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e)
        if (i + e < a.vocab) out[i + e] = f2bf(v[e]);
    }
  }
  __syncthreads();
  // the elements of the top tokens and of the target, once each
  if (tid < a.topk && idx[tid] >= 0) fix_up(a, idx, pk, tid, idx[tid], zt[tid] - m, target, gt, g1, out);
  if (tid == 0 && target >= 0) fix_up(a, idx, pk, a.topk, target, sh_z - m, target, gt, g1, out);
}

template <typename T, bool CE, Grad GRAD, Rows ROWS>
cudaError_t launch_stream(const T* z, __nv_bfloat16* dz, const DistillArgs& a, int rows, int ctas, int per,
                          cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const int rc = once_per_device(done, [] {
    return static_cast<int>(cudaFuncSetAttribute(distill_stream_kernel<T, CE, GRAD, ROWS>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem));
  });
  if (rc) return static_cast<cudaError_t>(rc);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = kStreamSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  set_priority_attr(attr[1], s);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // as many clusters as run at once (a cluster lives within one GPC, so large ones may leave SMs over)
  static PerDevice<kMaxCluster + 1> at_once;
  int clusters = 0;
  const cudaError_t e = at_once.get(ctas, [&](int* n) {
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms() / ctas * ctas));
    return cudaOccupancyMaxActiveClusters(n, distill_stream_kernel<T, CE, GRAD, ROWS>, &cfg);
  }, &clusters);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>((rows < clusters ? rows : clusters) * ctas));
  return cudaLaunchKernelEx(&cfg, distill_stream_kernel<T, CE, GRAD, ROWS>, z, dz, a, rows, ctas, per);
}

template <typename T, Grad GRAD, Rows ROWS>
cudaError_t launch_stream_ce(const T* z, __nv_bfloat16* dz, const DistillArgs& a, int rows, int ctas, int per,
                             cudaStream_t s) {
  return a.ce > 0.f ? launch_stream<T, true, GRAD, ROWS>(z, dz, a, rows, ctas, per, s)
                    : launch_stream<T, false, GRAD, ROWS>(z, dz, a, rows, ctas, per, s);
}
template <typename T, Grad GRAD>
cudaError_t launch_stream_rows(const T* z, __nv_bfloat16* dz, const DistillArgs& a, int rows, int ctas, int per,
                               bool aligned, cudaStream_t s) {
  if (!aligned) return launch_stream_ce<T, GRAD, kAny>(z, dz, a, rows, ctas, per, s);
  if (a.vocab * sizeof(T) % 16) return launch_stream_ce<T, GRAD, kAligned>(z, dz, a, rows, ctas, per, s);
  return launch_stream_ce<T, GRAD, kWhole>(z, dz, a, rows, ctas, per, s);
}

// Clusters of `ctas` for slices of at most `most` elements; with rows for less than
// half of the SMs, more of them a row, down to slices of `few`.
int row_ctas(int rows, int vocab, int64_t most, int64_t few) {
  int ctas = 1;
  while (ctas < kMaxCluster && most * ctas < vocab) ctas *= 2;
  while (ctas < kMaxCluster && static_cast<int64_t>(rows) * ctas * 2 <= num_sms() && few * ctas < vocab) ctas *= 2;
  return ctas;
}

constexpr int kShortBytes = 16384;

// Which kernel takes the rows:
//   up to 16 KB (where all rows are aligned for wide loads and stores) or 4096
//       elements   registers, in the fewest threads that keep 4 or 8 loads each (16
//       or 32 of one element).  With 64 slots and 64 threads 65536 rows of 512 fp32
//       take 234 us at 4 loads and 287 at 8, 8192 x 2048 take 84 with 256 x 4 and 46
//       with 64 x 8, 8192 x 4096 take 88 with 256 x 4, 78 with 64 x 16 and 67 with 128 x 8
//   longer         the stream: 2048 x 32000 fp32 76 us, 115 with the row in
//       registers; 2048 x 32001 bf16, unaligned, 81 us, 149 read twice, 1000 x
//       100001 fp32 141 and 280 (in registers; 350 read twice).  Unaligned bf16
//       rows of 8 to 16 KB are read twice: 8192 x 5001 130 us, 184 in the stream
//   what no cluster of 8 holds   is read twice
template <typename T, bool VEC>
cudaError_t launch_rows(const T* z, __nv_bfloat16* dz, const DistillArgs& a, int rows, bool aligned, bool wide,
                        cudaStream_t s) {
  constexpr int kFew = VEC ? 4 : 16, kMore = VEC ? 8 : 32;  // loads a thread
  if (a.vocab <= Slice<T, VEC, kFew, 64>::kElems)
    return launch_k(distill_row_kernel<T, VEC, kFew, 64>, rows, 64, 0, s, z, dz, a);
  if (a.vocab <= Slice<T, VEC, kMore, 64>::kElems)
    return launch_k(distill_row_kernel<T, VEC, kMore, 64>, rows, 64, 0, s, z, dz, a);
  if (a.vocab <= Slice<T, VEC, kMore, 128>::kElems)
    return launch_k(distill_row_kernel<T, VEC, kMore, 128>, rows, 128, 0, s, z, dz, a);
  // without dz a slice need not fit in the ring: 1000 x 200000 bf16 take 87 us in one slice, 178 in four
  const int64_t most = dz ? kMaxSliceChunks * kChunk / static_cast<int>(sizeof(T)) : a.vocab;
  const int ctas = row_ctas(rows, a.vocab, most, kShortBytes / static_cast<int>(sizeof(T)));
  if (most * ctas < a.vocab || (!VEC && a.vocab * sizeof(T) <= kShortBytes))
    return launch_k(distill_kernel<T, VEC>, rows, kDistillThreads, 0, s, z, dz, a);
  const int per = ((a.vocab + ctas - 1) / ctas + 7) & ~7;
  if (!dz) return launch_stream_rows<T, kLoss>(z, dz, a, rows, ctas, per, aligned, s);
  if (wide) return launch_stream_rows<T, kWide>(z, dz, a, rows, ctas, per, aligned, s);
  return launch_stream_ce<T, kSingle, kAny>(z, dz, a, rows, ctas, per, s);
}

}  // namespace

int launch_distill(int dtype, int rows, int vocab, const void* logits, int64_t ld, int topk, const int32_t* top_idx,
                   const float* top_logit, float temperature, float kd_scale, int seq, const int32_t* tokens, int row0,
                   float ce_scale, float* loss_rows, void* dz, int64_t lddz, cudaStream_t s) {
  if (dtype != DT_F32 && dtype != DT_BF16) return set_error(GPIPE_ERR_UNSUPPORTED, "distill: dtype must be 0 or 1");
  if (rows < 1 || rows > (1 << 27) || vocab < 1 || vocab > (1 << 30) || ld < vocab || topk < 1 || topk > kMaxTop)
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "distill: need 1 <= rows <= 2^27, 1 <= vocab <= 2^30, ld >= vocab and 1 <= topk <= %d", kMaxTop);
  if (!(temperature > 0.f) || !(temperature < INFINITY) || !(kd_scale >= 0.f) || !(kd_scale < INFINITY) ||
      !(ce_scale >= 0.f) || !(ce_scale < INFINITY))
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: need a finite temperature > 0 and finite scales >= 0");
  // (from 2^-126 on log2(e) / T, the kernels' factor, is finite too)
  if (temperature < FLT_MIN || !(kd_scale * temperature * temperature < INFINITY))
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "distill: the temperature must be at least 2^-126 and kd_scale temperature^2 finite in fp32");
  if (!logits || !top_idx || !top_logit || !loss_rows)
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: NULL logits, top_idx, top_logit or loss_rows");
  if (ce_scale > 0.f && (!tokens || seq < 1 || row0 < 0))
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: ce_scale > 0 needs tokens, seq >= 1 and row0 >= 0");
  const size_t es = dtype == DT_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(logits) % es) || (reinterpret_cast<uintptr_t>(dz) % 2) || !attn::al4(top_idx) ||
      !attn::al4(top_logit) || !attn::al4(loss_rows) || (ce_scale > 0.f && !attn::al4(tokens)))
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: tensors must be aligned to their elements");
  if (dz && lddz < vocab) return set_error(GPIPE_ERR_INVALID_ARG, "distill: lddz must be at least vocab");
  using attn::overlaps;
  using attn::Range;
  const size_t nr = static_cast<size_t>(rows);
  const Range in = {logits, ((nr - 1) * ld + vocab) * es}, out = {dz, dz ? ((nr - 1) * lddz + vocab) * 2 : 0};
  const bool in_place = overlaps(out, {in});
  if (in_place && !(dz == logits && (rows == 1 || lddz * 2 == ld * static_cast<int64_t>(es))))
    return set_error(GPIPE_ERR_INVALID_ARG,
                     "distill: dz overlaps the logits, which needs the same address and the same row stride in bytes");
  // the tokens that are read: the last row's only if it has a target
  Range labels = {nullptr, 0};
  if (ce_scale > 0.f) labels = {tokens + row0 + 1, (nr - ((static_cast<int64_t>(row0) + rows) % seq == 0)) * 4};
  const Range idx = {top_idx, nr * topk * 4}, val = {top_logit, nr * topk * 4}, loss = {loss_rows, nr * 4};
  if (overlaps(loss, {in, out, idx, val, labels}) || overlaps(out, {idx, val, labels}))
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: loss_rows and dz may not overlap each other or the other inputs");
  DistillArgs a;
  a.vocab = vocab;
  a.topk = topk;
  a.seq = seq;
  a.row0 = row0;
  a.ld = ld;
  a.lddz = lddz;
  a.top_idx = top_idx;
  a.top_logit = top_logit;
  a.tokens = tokens;
  a.inv_t = 1.f / temperature;
  a.kd = kd_scale * temperature * temperature;
  a.kd_grad = kd_scale * temperature;
  a.ce = ce_scale;
  a.loss = loss_rows;
  a.err = device_error_ptr();
  a.in_place = in_place;
  if (!a.err) return set_error(GPIPE_ERR_CUDA, "distill: no device error word");
  const int64_t vec_elems = 16 / static_cast<int64_t>(es);
  // where a row of logits meets a 16-byte boundary, its dz is aligned for the stores of as many elements
  const bool wide = (lddz - ld) % vec_elems == 0 &&
                    (reinterpret_cast<uintptr_t>(dz) / 2 - reinterpret_cast<uintptr_t>(logits) / es) % vec_elems ==
                        0;
  const bool aligned = al16(logits) && (rows == 1 || ld % vec_elems == 0);
  // rows whose every start is aligned for 16-byte loads and the stores that go with them
  const bool vec = aligned && ld % vec_elems == 0 &&
                   (!dz || (reinterpret_cast<uintptr_t>(dz) % (es == 4 ? 8 : 16) == 0 && lddz % vec_elems == 0));
  __nv_bfloat16* d = static_cast<__nv_bfloat16*>(dz);
  auto launch = [&](auto* z) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(z)>>;
    return vec ? launch_rows<T, true>(z, d, a, rows, aligned, wide, s)
               : launch_rows<T, false>(z, d, a, rows, aligned, wide, s);
  };
  cudaError_t e = dtype == DT_F32 ? launch(static_cast<const float*>(logits))
                                  : launch(static_cast<const __nv_bfloat16*>(logits));
  count_launch();
  const cudaError_t last = cudaGetLastError();
  if (e == cudaSuccess) e = last;
  if (e != cudaSuccess) return set_error(GPIPE_ERR_CUDA, "distill launch: %s", cudaGetErrorString(e));
  return GPIPE_OK;
}

}  // namespace gp
