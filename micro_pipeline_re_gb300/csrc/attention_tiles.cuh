// What the attention kernels share: constants of the 64-wide head, the swizzled
// shared-memory tiles, tensor-memory row access, bounded waits, and the tensor
// map encoder.
//
// Shared-memory tiles (1024-B aligned, 128-B rows, 16-B unit u of row r at
// r*128 + ((u ^ (r&7)) * 16)):
//   as a K-major operand (rows = M or N, 64 head columns or 64 keys per row):
//     the 16-wide k slice kk starts 32*kk bytes into each row; 8-row groups
//     are 1024 B apart;
//   as an MN-major operand (rows = K, 64 head columns = N per row): the
//     16-deep k slice kk starts 2048*kk bytes further.
#pragma once
#include <cuda.h>

#include <atomic>
#include <initializer_list>

#include "common.cuh"

namespace gp {
namespace attn {

constexpr int HD = 64;                                      // head width
constexpr float kScaleLog2 = 0.125f * 1.4426950408889634f;  // scale * log2(e)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int T128 = 128 * 128;  // bytes of a 128-row tile (128 B per row)
constexpr int T64 = 64 * 128;    // bytes of a 64-row tile

__device__ __forceinline__ uint32_t swz(int r, int u) { return static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4)); }
// K-major operand tile, 16-wide k slice kk (0..3)
__device__ __forceinline__ uint64_t kdesc(uint32_t tile, int kk) { return sw128_desc(tile + kk * 32, 16, 1024); }
// MN-major operand tile (64 wide), 16-deep k slice kk
__device__ __forceinline__ uint64_t mndesc(uint32_t tile, int kk) { return sw128_desc(tile + kk * 2048, 8192, 1024); }

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Load 32 fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void ld_row32(uint32_t taddr, float* v) {
  uint32_t u[32];
  tmem_ld32(taddr, u);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
}

// Load 32 * N fp32 columns of this thread's lane from the column addresses
// a[0..N-1]: every load is issued before the one wait, so their latencies
// overlap (a TMEM load takes a few hundred cycles to return).
template <int N>
__device__ __forceinline__ void ld_rows(const uint32_t* a, float* v) {
  uint32_t u[32 * N];
#pragma unroll
  for (int c = 0; c < N; ++c) tmem_ld32(a[c], u + 32 * c);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32 * N; ++i) v[i] = __uint_as_float(u[i]);
}


// Write 32 values of row r as bf16 into a swizzled tile at units u0..u0+3.
__device__ __forceinline__ void st_row32_bf16(uint8_t* tile, int r, int u0, const float* v) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint4 w;
    w.x = pack_bf16x2(v[8 * u + 0], v[8 * u + 1]);
    w.y = pack_bf16x2(v[8 * u + 2], v[8 * u + 3]);
    w.z = pack_bf16x2(v[8 * u + 4], v[8 * u + 5]);
    w.w = pack_bf16x2(v[8 * u + 6], v[8 * u + 7]);
    *reinterpret_cast<uint4*>(tile + swz(r, u0 + u)) = w;
  }
}

// Store 64 fp32 TMEM columns of this thread's lane, times scale, as bf16 to
// dst when `valid`.  Every thread of the warp calls it (the TMEM loads are
// warp-collective); only the stores depend on `valid`.
__device__ __forceinline__ void store_row64(uint32_t taddr, __nv_bfloat16* dst, float scale, bool valid) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[32];
    ld_row32(taddr + 32 * h, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= scale;
    if (valid) {
#pragma unroll
      for (int u = 0; u < 4; ++u) store8(dst + 32 * h + 8 * u, v + 8 * u);
    }
  }
}

// Bounded wait that gives up at once after any earlier give-up in the CTA.
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* abort) {
  if (*abort) return false;
  if (mbar_wait_bounded(bar, parity, err, code)) return true;
  *abort = 1;
  return false;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<EncodeFn>(p);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A tensor's bytes, for the checks of outputs against the other tensors of a call.
struct Range {
  const void* at;
  size_t bytes;  // 0 where the call has no such tensor
};
inline bool overlaps(Range out, std::initializer_list<Range> others) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(out.at);
  for (const Range& r : others) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(r.at);
    if (out.bytes && r.bytes && a < b + r.bytes && b < a + out.bytes) return true;
  }
  return false;
}

}  // namespace attn
}  // namespace gp
