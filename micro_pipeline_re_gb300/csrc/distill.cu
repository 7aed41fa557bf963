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
// Both softmaxes share the maximum m of z: q_T = e^{(z - m) / T} / s_T.  The
// subtraction comes first, so the exponent is exact to fp32 however large the
// logits are.  The top tokens are few, so dz is written as if there were none
// and their elements are written again; slots that name the same token are
// added by the first of them, in slot order, so that nothing depends on timing.
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

  int target = -1;
  if (a.ce > 0.f) {
    const int64_t g = a.row0 + r;
    if (g % a.seq != a.seq - 1) {
      target = a.tokens[g + 1];
      if (target < 0 || target >= a.vocab) {
        if (tid == 0) atomicExch(a.err, DERR_BAD_TOKEN);
        target = -1;
      }
    }
  }
  if (tid < a.topk) {
    int i = a.top_idx[r * a.topk + tid];
    if (i >= a.vocab) {
      atomicExch(a.err, DERR_BAD_TOKEN);
      i = -1;
    }
    idx[tid] = i;
    tl[tid] = i >= 0 ? a.top_logit[r * a.topk + tid] * a.inv_t : -INFINITY;
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
    // teacher: p over the filled slots
    float tm = -INFINITY;
    for (int k = lane; k < a.topk; k += 32) tm = fmaxf(tm, tl[k]);
    tm = warp_max(tm);
    const float tb = tm == -INFINITY ? 0.f : tm;
    float ts = 0.f;
    for (int k = lane; k < a.topk; k += 32) ts += expf(tl[k] - tb);
    ts = warp_sum(ts);
    const float log_ts = logf(ts), log_st = logf(st);
    float kl = 0.f;
    for (int k = lane; k < a.topk; k += 32) {
      const float p = ts == 0.f ? 0.f : expf(tl[k] - tb) / ts;
      pk[k] = p;
      if (p != 0.f) kl += p * ((tl[k] - tb - log_ts) - ((zt[k] - m) * a.inv_t - log_st));
    }
    kl = warp_sum(kl);
    if (lane == 0) {
      sh[0] = m;
      sh[1] = s1;
      sh[2] = st;
      sh_has = ts == 0.f ? 0.f : 1.f;
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
  const bool slot = tid < a.topk && idx[tid] >= 0;
  if (slot || (tid == a.topk && target >= 0)) {
    const int me = slot ? idx[tid] : target;
    const float x = (slot ? zt[tid] : sh_z) - m;
    float p = 0.f;
    bool first = true;
    for (int k = 0; k < a.topk; ++k)
      if (idx[k] == me) {
        if (k < tid) first = false;
        p += pk[k];
      }
    if (first) {
      float g = gt != 0.f ? ex2_approx(x * ct) * gt - a.kd_grad * p : 0.f;
      if (g1 != 0.f) g += ex2_approx(x * c1) * g1;
      if (me == target) g -= a.ce;
      out[me] = f2bf(g);
    }
  }
}

}  // namespace

int launch_distill(int dtype, int rows, int vocab, const void* logits, int64_t ld, int topk, const int32_t* top_idx,
                   const float* top_logit, float temperature, float kd_scale, int seq, const int32_t* tokens, int row0,
                   float ce_scale, float* loss_rows, void* dz, int64_t lddz, cudaStream_t s) {
  if (dtype != DT_F32 && dtype != DT_BF16) return set_error(GPIPE_ERR_UNSUPPORTED, "distill: dtype must be 0 or 1");
  if (rows < 1 || vocab < 1 || ld < vocab || topk < 1 || topk > kMaxTop)
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: need rows, vocab >= 1, ld >= vocab and 1 <= topk <= %d", kMaxTop);
  if (!(temperature > 0.f) || !(temperature < INFINITY) || !(kd_scale >= 0.f) || !(kd_scale < INFINITY) ||
      !(ce_scale >= 0.f) || !(ce_scale < INFINITY))
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: need a finite temperature > 0 and finite scales >= 0");
  if (!logits || !top_idx || !top_logit || !loss_rows)
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: NULL logits, top_idx, top_logit or loss_rows");
  if (ce_scale > 0.f && (!tokens || seq < 1 || row0 < 0))
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: ce_scale > 0 needs tokens, seq >= 1 and row0 >= 0");
  const size_t es = dtype == DT_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(logits) % es) || (reinterpret_cast<uintptr_t>(dz) % 2))
    return set_error(GPIPE_ERR_INVALID_ARG, "distill: logits and dz must be aligned to their elements");
  bool in_place = false;
  if (dz) {
    if (lddz < vocab) return set_error(GPIPE_ERR_INVALID_ARG, "distill: lddz must be at least vocab");
    const uintptr_t zb = reinterpret_cast<uintptr_t>(logits), db = reinterpret_cast<uintptr_t>(dz);
    const uintptr_t ze = zb + (static_cast<uintptr_t>(rows - 1) * ld + vocab) * es;
    const uintptr_t de = db + (static_cast<uintptr_t>(rows - 1) * lddz + vocab) * 2;
    in_place = zb < de && db < ze;
    if (in_place && !(zb == db && (rows == 1 || lddz * 2 == ld * static_cast<int64_t>(es))))
      return set_error(GPIPE_ERR_INVALID_ARG,
                       "distill: dz overlaps the logits, which needs the same address and the same row stride in bytes");
  }
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
  // rows whose every start is aligned for 16-byte loads (and the stores that go with them)
  const bool vec = al16(logits) && ld * static_cast<int64_t>(es) % 16 == 0 &&
                   (!dz || (reinterpret_cast<uintptr_t>(dz) % (es == 4 ? 8 : 16) == 0 && lddz % (es == 4 ? 4 : 8) == 0));
  __nv_bfloat16* d = static_cast<__nv_bfloat16*>(dz);
  if (dtype == DT_F32) {
    const float* z = static_cast<const float*>(logits);
    (void)launch_k(vec ? distill_kernel<float, true> : distill_kernel<float, false>, rows, kDistillThreads, 0, s, z, d, a);
  } else {
    const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(logits);
    (void)launch_k(vec ? distill_kernel<__nv_bfloat16, true> : distill_kernel<__nv_bfloat16, false>, rows,
                   kDistillThreads, 0, s, z, d, a);
  }
  count_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(GPIPE_ERR_CUDA, "distill launch: %s", cudaGetErrorString(e));
  return GPIPE_OK;
}

}  // namespace gp
