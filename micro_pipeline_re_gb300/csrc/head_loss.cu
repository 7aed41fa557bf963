// The head's loss without the logits: next-token cross-entropy of h E^T over the
// tied matrix E, and its gradients with respect to h and E, made for a piece of
// the vocabulary at a time.
//
//   z = h_r E^T (limited to [-clip, clip]),  p = softmax(z)
//   loss_r = -w_r a log p_t,                 a = inv_count
//   g = w_r (p - onehot(t)),                 dh = a g E,  dE = a g^T h
//
// Launches:
//      head_copy_kernel           (large calls whose h is not on 32-byte rows) a copy
//   1  head_gemm_kernel<kStats>   z tile by tile in tensor memory; of every row and
//                                 128 columns only (rho, sum 2^{z log2 e - rho}) leaves.
//                                 With gradients, the first piece's powers go to where
//                                 its g will be (fp16).  Up to 64 rows without gradients:
//      head_gemm_kernel<kFew>     the same with the vocabulary as the products' rows
//   2  head_rows_kernel           joins them, the loss, and what 3 needs of a row
//   3  head_scale_kernel          the first piece's g from the powers, in place
//      head_gemm_kernel<kGrad>    or z again, turned into g in the epilogue
//   per piece of the vocabulary:
//   4  head_gemm_kernel<kProducts>  both products of g, tiles of dh and of dE in one
//                                 launch, and the next piece's g, so that one's last
//                                 round fills the other's
//   5  head_dh_kernel             sums of dh over pieces and parts of K into bf16
//
// Arithmetic.  Exponentials are powers of two, with an integer reference rho of each
// row: the argument fma(z, log2 e, -rho) is rounded once, and sums move from one
// reference to another exactly.  The target's column is left out of the sums, and its
// logit is a dot product of its own in fp32 (tensor cores truncate as they add: 1024
// terms left z_t up to 2e-5 short, which showed in the loss; this way 1e-7).  So
//   loss = log1p(sum_{v != t} e^{z_v - z_t}),  g_t = -w sum_{v != t} p_v
// keep their digits where p_t is close to 1 (dh, and dE of up to 64 rows, get back what g_t
// loses to its rounding, which would be an error of a whole row).  g is rounded to bf16, relative to
// each value, as gpipe_op_cross_entropy rounds its dz; inv_count multiplies the
// finished fp32 sums, so that g_t, close to -w for most rows, is close to a whole number
// and its rounding does not add up over the rows.
//
// Cost: 8 rows vocab d flops with both gradients, 6 for a first piece whose powers are kept.
// Memory: 2 B an element of a piece of g, or of two where there are several, which is all
// that is ever held of the logits.  The powers are fp16 because it has three bits more than
// bf16, 2^-28 of the largest of 128 down (their reference puts that near 2^14): g's rounding
// to bf16 stays the only one that tells.
//
// Measured at 2048 rows x 1024 x 32000 (134 GFLOP a product; ncu, and 291 us for all five in
// a graph, 317 in a row, where the GPU meets its power limit): kStats 83 us with the powers
// and 74 without (1805 TFLOP/s, 92 % of a library product's burst rate; tensor pipe 77 %
// active), head_rows 5, head_scale 42 (262 MB, 6.3 TB/s), kProducts 149 (1802 TFLOP/s, tensor
// pipe 87 %), head_dh 7.  An issuing thread whose waits read no clock unless they have to
// took kStats from 88 us to 78.  Below 512 columns of h the epilogue bounds the first pass:
// 1.6 us a 256 x 256 tile, whatever d.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <utility>

#include "../../include/gpipe.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_util.cuh"

namespace gp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct HeadArgs {
  int rows, d, vocab, seq, row0;
  const int32_t* tokens;
  const float* weight;
  float inv_count, clip;
};

// What the gradient pass knows of a row: the reference and w / sum e^{z - ...} for
// p, g of the target's column, and the target (-1: the row has none).
struct HeadRow {
  float rho, scale, gt;
  int target;
};

// Target of row r, or -1 (none: the end of a sequence, a negative id, weight 0).
__device__ __forceinline__ int head_target(const HeadArgs& a, int r, float& w, int* err) {
  w = a.weight ? a.weight[r] : 1.f;
  const unsigned at = static_cast<unsigned>(a.row0) + static_cast<unsigned>(r);
  if (w == 0.f || at % static_cast<unsigned>(a.seq) == static_cast<unsigned>(a.seq) - 1u) return -1;
  const int t = a.tokens[at + 1];
  if (t >= a.vocab && err) atomicExch(err, DERR_BAD_TOKEN);
  return t >= 0 && t < a.vocab ? t : -1;
}

// What a number loses to its rounding to bf16.
__device__ __forceinline__ float lost(float x) { return x - bf2f(f2bf(x)); }

__device__ __forceinline__ float limit(float z, float c) {  // keeps NaN
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n\tmin.NaN.f32 %0, %0, %3;" : "=&f"(y) : "f"(z), "f"(-c), "f"(c));
  return y;
}

// ---------------------------------------------------------------------------
// The products: persistent, a pair of CTAs (cluster of two) per 256 x 256 tile.
//   warp 0 / lane 0   copies through a ring of stages, each CTA its 128 rows of A and
//                     128 columns of B of a k-block of 64; both complete on rank 0's
//                     barrier
//   warp 1 / lane 0 of rank 0   issues 256-row products into one of two accumulators
//   warps 2..9        epilogue, each on its own: 32 rows, 128 columns, 32 at a time
// (the organisation of the library's persistent GEMM on SM pairs).
// ---------------------------------------------------------------------------
enum Mode { kStats, kFew, kGrad, kProducts };
enum DhOut { kDhStore, kDhAdd, kDhBf16 };  // fp32, fp32 added, bf16 and final

constexpr int kTile = 256;     // rows and columns of a pair's tile
// kFew: rows of h, its columns.  A tile of kStats costs 256 rows' products however few there
// are: 1 row over 32000 x 1024 (65 MB, here from the L2) 18.4 us this way, 26.6 that way; 64
// rows 16.3 and 18.1
constexpr int kFewRows = 64;
constexpr int kK = 64;         // a k-block
constexpr int kHeadThreads = 320;
constexpr int kGroup = 16;     // row tiles that the tiles in flight share
// d from which reading the first piece's powers is cheaper than making z again: with both
// gradients over 32000 columns 2048 rows take 187 us kept and 181 made again at d = 512, 242
// and 243 at 768, 291 and 314 at 1024; 512 rows 68 and 67, 83 and 84, 98 and 102
constexpr int kKeepWidth = 768;
// rows x vocab x d from which h is copied where its rows do not start on 32 bytes, the L2's
// sectors: 2048 x 712 x 32000, the loss, take 75 us as it is and 62 with the copy (720 columns 60),
// 2048 x 1016 96 and 82 (1024 columns 75).  That E's rows lie like that hardly tells.
constexpr int64_t kCopyWork = int64_t{1} << 33;
constexpr int kWideRows = 1216;  // rows up to which each has a CTA to join its sums (eight an SM)
constexpr int kPlanPairs = 76; // pairs of SMs that the split of dh's K is planned for (any number runs it)

template <Mode MODE>
struct HeadCfg {
  static constexpr int kColumns = MODE == kFew ? kFewRows : kTile;  // of a pair's tile
  static constexpr int kA = 128 * kK * 2;                           // bytes of the operands of a CTA's stage
  static constexpr int kB = kColumns / 2 * kK * 2;
  static constexpr int kStage = kA + kB;
  // 32 x 32 elements leaving (kFew: being turned round)
  static constexpr int kBox = MODE == kProducts ? 4096 : (MODE == kFew ? 32 * 33 * 2 : 2048);
  static constexpr int kStages = MODE == kProducts ? 5 : (MODE == kFew ? 9 : 6);
  static constexpr int kOffBox = kStages * kStage;
  static constexpr int kOffBar = kOffBox + 8 * 2 * kBox;
  static constexpr int kSmem = 1024 + kOffBar + 512;
  static_assert(kOffBar % 8 == 0 && kSmem <= 232448, "over the shared memory of a CTA");
};

struct HeadMaps {
  CUtensorMap a, b;    // logits: h and the piece of E; products: g and the piece of E (dh)
  CUtensorMap c;       // where the tiles leave to: g, or dh
  CUtensorMap a2, b2, c2;  // products: g the other way round and h (dE), dE
  CUtensorMap a3, b3, c3;  // products: h, the next piece of E and its g
};

// A list of n tiles shared out to the pairs: those from `late` on, which have less to do
// before it, take `ahead` each, then all take the others in turn.
struct Share {
  int n, late, ahead;
  __device__ __forceinline__ int tile(int j, int pair, int pairs) const {  // a pair's j-th; n or more: none
    const int rest = pairs - late, mine = pair >= late ? ahead : 0;
    return j < mine ? j * rest + (pair - late) : ahead * rest + (j - mine) * pairs + pair;
  }
};

struct HeadGemm {
  HeadArgs row;
  int cols;              // columns of the piece
  int v0;                // its first
  int m_tiles, n_tiles;  // logits: rows x columns; products: dh's rows x d
  float2* parts;         // kStats: [rows][2 n_tiles]
  int keep;              // kStats: columns whose powers go to g (fp16)
  const HeadRow* info;   // kGrad, and kProducts where its dh is final
  const __nv_bfloat16* emb;
  // kProducts
  const __nv_bfloat16* hm;  // the rows that dE is made of
  int64_t ldm;
  int splits, rows_pad;  // parts of dh's K, each with a buffer of rows_pad rows
  int dh_items, dh_out;
  Share de, g;              // tiles of dE and of the next piece's g
  bool de_f32;
  int g_tiles, g_cols, g_v0;  // the next piece's tiles across, columns and first column
};

enum Kind { kLogits, kDh, kDe };
struct Item {
  int m0, n0, k0, nk;  // origin of the tile; first k-block and their number
  int split;
  Kind kind;
};

// The tiles of a pair, in order.  Logits: every pairs-th of the grouped tile order
// (row tiles fastest within a group, so the tiles in flight share bands of both operands).
// Products: its share of dh's tiles, which are few and long, then of dE's and of the next
// piece's g.
template <Mode MODE>
struct Walk {
  int pair, pairs, i = 0, j = 0, k = 0;
  __device__ Walk(int p, int n) : pair(p), pairs(n) {}
  // tile t of a grid whose row tiles are fastest within groups of kGroup
  __device__ __forceinline__ void logits(const HeadGemm& a, int t, int n_tiles, Item& it) {
    const int per_group = kGroup * n_tiles;
    const int grp = t / per_group, r = t - grp * per_group, first = grp * kGroup;
    const int gm = min(kGroup, a.m_tiles - first);
    it.m0 = (first + r % gm) * kTile;
    it.n0 = (r / gm) * kTile;
    it.nk = (a.row.d + kK - 1) / kK;
    it.kind = kLogits;
  }
  __device__ __forceinline__ bool next(const HeadGemm& a, Item& it) {
    it.split = 0;
    it.k0 = 0;
    if (MODE != kProducts) {
      const int t = pair + i++ * pairs;
      if (t >= a.m_tiles * a.n_tiles) return false;
      logits(a, t, a.n_tiles, it);
      return true;
    }
    const int t = pair + i * pairs;
    if (t < a.dh_items) {
      ++i;
      const int n = t % a.n_tiles, m = t / a.n_tiles % a.m_tiles;
      it.split = t / (a.n_tiles * a.m_tiles);
      const int nk = (a.cols + kK - 1) / kK;
      it.m0 = m * kTile;
      it.n0 = n * kTile;
      it.k0 = static_cast<int>(static_cast<int64_t>(nk) * it.split / a.splits);
      it.nk = static_cast<int>(static_cast<int64_t>(nk) * (it.split + 1) / a.splits) - it.k0;
      it.kind = kDh;
      return true;
    }
    const int e = a.de.tile(j, pair, pairs);
    if (e >= a.de.n) {
      const int g = a.g.tile(k++, pair, pairs);
      if (g >= a.g.n) return false;
      logits(a, g, a.g_tiles, it);
      return true;
    }
    ++j;
    it.kind = kDe;
    it.m0 = e / a.n_tiles * kTile;
    it.n0 = e % a.n_tiles * kTile;
    it.nk = (a.row.rows + kK - 1) / kK;
    return true;
  }
};

// Byte offset of 16-byte unit u of row r of a 32 x 32 box, as the tensor maps swizzle
// it: 64-byte rows (bf16) or 128-byte rows (fp32).
__device__ __forceinline__ uint32_t box_bf16(int r, int u) {
  return static_cast<uint32_t>(r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
}
__device__ __forceinline__ uint32_t box_f32(int r, int u) {
  return static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4));
}
__device__ __forceinline__ void wait_read_1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t u) {
  float2 f;
  asm("{\n .reg .f16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(u));
  return f;
}

// Arrival at a barrier of the pair without the release of earlier writes, which costs
// about 1200 clocks at cluster scope.  No writes are handed over: each lane's loads of the
// tensor memory have completed (tcgen05.wait::ld) and are ordered before what follows by its
// tcgen05.fence::before_thread_sync, the lanes' before this one lane's arrival by __syncwarp(),
// and the products behind the issuer's wait by its tcgen05.fence::after_thread_sync.  Generic
// memory that a warp wrote before is not visible through it, and nobody reads any by it.
__device__ __forceinline__ void arrive_relaxed(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// Bounded wait; CLUSTER: for arrivals from the peer CTA, too.  The hint lets the hardware
// put the warp aside for up to 20 us a try, so that it does not poll beside the others.
// Gives up at once after any earlier give-up in the CTA.
template <bool CLUSTER = false>
__device__ __forceinline__ bool try_wait_long(uint32_t at, uint32_t parity) {
  uint32_t ok;
  if (CLUSTER)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(at), "r"(parity), "r"(20000u)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(at), "r"(parity), "r"(20000u)
        : "memory");
  return ok != 0;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool head_wait(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* abort) {
  const uint32_t at = smem_u32(bar);
  if (try_wait_long<CLUSTER>(at, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
#pragma unroll 1
  while (!try_wait_long<CLUSTER>(at, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicExch(err, code);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// N logits v of a row become the powers 2^{v log2 e - rho}, at most 2^14; their sum.
template <int N>
__device__ __forceinline__ float to_powers(float* v, float& rho) {
  float m8[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m8[j] = fmaxf(v[j], v[j + 8]);
#pragma unroll
    for (int k = 16; k < N; k += 16) m8[j] = fmax3(m8[j], v[j + k], v[j + k + 8]);
  }
  const float m = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
  rho = ceilf(m * kLog2e) - 14.f;
  // (-inf: nothing but columns that are left out, powers of 0 whatever the reference)
  const float at = rho == -INFINITY ? 0.f : rho;
  const f32x2 l2 = pack2(kLog2e, kLog2e), ref = pack2(-at, -at);
  f32x2 sum[8];
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    float x, y;
    unpack2(fma2(pack2(v[j], v[j + 1]), l2, ref), x, y);
    v[j] = ex2_approx(x);
    v[j + 1] = ex2_approx(y);
    const f32x2 e = pack2(v[j], v[j + 1]);
    sum[(j >> 1) & 7] = j < 16 ? e : add2(sum[(j >> 1) & 7], e);
  }
  float x, y;
  unpack2(add2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), add2(add2(sum[4], sum[5]), add2(sum[6], sum[7]))), x,
          y);
  return x + y;
}

template <Mode MODE>
__global__ void __launch_bounds__(kHeadThreads, 1)
    head_gemm_kernel(const __grid_constant__ HeadMaps maps, const HeadGemm a, int* err) {
  using Cfg = HeadCfg<MODE>;
  constexpr int STAGES = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBar);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;  // accumulator b holds a finished tile
  uint64_t* acce = accf + 2;        // accumulator b has been drained
  uint64_t* bfin = acce + 2;        // every product of the pair has completed
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bfin + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank() & 1u);
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 16);  // the epilogue warps of both CTAs
    }
    mbar_init(bfin, 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tslot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before any copy or arrival names them
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // global memory from here on.  The gradient pass's products read only h (or its copy) and
  // E, which were there before the stats kernel's wait ended and which no launch behind that
  // wait writes (each lets the next one start only after its own wait, or after that of the
  // stats kernel); its epilogue waits for what it reads, the rows, and for the readers of
  // what it writes.
  if (MODE != kGrad) griddep_wait();

  Walk<MODE> walk(pair, pairs);
  Item it;
  if (warp == 0) {
    if (lane == 0) {
      int n = 0, s = 0;  // k-blocks so far; the stage of the next, whose ring has been round `turn` times (mod 2)
      uint32_t turn = 0;
      const uint32_t full_leader = map_peer(smem_u32(full), 0);
      while (!*abort && walk.next(a, it)) {
        const int am = it.m0 + rank * 128, bn = it.n0 + rank * (Cfg::kColumns / 2);
        for (int kb = 0; kb < it.nk; ++kb, ++n) {
          if (!head_wait(&empty[s], turn ^ 1, err, DERR_TMA_WAIT, abort)) break;
          uint8_t* sa = smem + s * Cfg::kStage;
          uint8_t* sb = sa + Cfg::kA;
          const int k = (it.k0 + kb) * kK;
          const uint32_t fb = full_leader + s * 8;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * Cfg::kStage);
          if (MODE != kProducts) {
            tma_load_2d_pair(sa, &maps.a, k, am, fb);
            tma_load_2d_pair(sb, &maps.b, k, bn, fb);
          } else if (it.kind == kLogits) {
            tma_load_2d_pair(sa, &maps.a3, k, am, fb);
            tma_load_2d_pair(sb, &maps.b3, k, bn, fb);
          } else if (it.kind == kDh) {
            tma_load_2d_pair(sa, &maps.a, k, am, fb);
            tma_load_2d_pair(sb, &maps.b, bn, k, fb);
            tma_load_2d_pair(sb + 8192, &maps.b, bn + 64, k, fb);
          } else {
            tma_load_2d_pair(sa, &maps.a2, am, k, fb);
            tma_load_2d_pair(sa + 8192, &maps.a2, am + 64, k, fb);
            tma_load_2d_pair(sb, &maps.b2, bn, k, fb);
            tma_load_2d_pair(sb + 8192, &maps.b2, bn + 64, k, fb);
          }
          if (++s == STAGES) {
            s = 0;
            turn ^= 1;
          }
        }
      }
      // no copy may still be landing in shared memory when a CTA of the pair leaves
      if (rank == 0)
        for (int j = (n > STAGES ? n - STAGES : 0); j < n; ++j)
          mbar_wait_bounded(&full[j % STAGES], (j / STAGES) & 1, err, DERR_DRAIN_WAIT);
    }
    griddep_launch();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int i = 0, s = 0;
      uint32_t turn = 0;
      const uint32_t stages = smem_u32(smem);
      for (; walk.next(a, it); ++i) {
        const int b = i & 1;
        if (!head_wait<true>(&acce[b], ((i >> 1) & 1) ^ 1, err, DERR_MMA_WAIT, abort)) break;
        tc_fence_after();
        const bool a_mn = MODE == kProducts && it.kind == kDe, b_mn = MODE == kProducts && it.kind != kLogits;
        const uint32_t idesc = a_mn   ? mma_idesc_bf16(kTile, kTile, true, true)
                               : b_mn ? mma_idesc_bf16(kTile, kTile, false, true)
                                      : mma_idesc_bf16(kTile, Cfg::kColumns, false, false);
        // descriptors but for the address, and their steps over 16 k (in units of 16 bytes): one
        // thread issues a k-block's four products in the 0.3 us that they take
        const uint64_t a_form = a_mn ? sw128_desc(0, 8192, 1024) : sw128_desc(0, 16, 1024),
                       b_form = b_mn ? sw128_desc(0, 8192, 1024) : sw128_desc(0, 16, 1024);
        const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
        const uint32_t acc = tmem + b * kTile;
        for (int kb = 0; kb < it.nk; ++kb) {
          if (!head_wait(&full[s], turn, err, DERR_MMA_WAIT, abort)) break;
          tc_fence_after();
          const uint32_t at = (stages + s * Cfg::kStage) >> 4;
#pragma unroll
          for (int kk = 0; kk < kK / 16; ++kk)
            tc_mma_f16_pair(acc, a_form + (at + kk * a_step), b_form + (at + (Cfg::kA >> 4) + kk * b_step), idesc,
                            (kb | kk) != 0 ? 1u : 0u);
          tc_commit_pair(&empty[s], 3);  // both CTAs' stage s is free again
          if (++s == STAGES) {
            s = 0;
            turn ^= 1;
          }
        }
        tc_commit_pair(&accf[b], 3);
      }
      tc_commit_pair(bfin, 1);
      mbar_wait_bounded(bfin, 0, err, DERR_DRAIN_WAIT);
    }
    griddep_launch();
  } else {
    if (MODE == kGrad) griddep_wait();
    // With few rows a row of dE is mostly one target's, and would show its rounding: it gets
    // back what g_t lost, too.  Lane l knows the targets of rows l and l + 32.  (For more rows
    // the search costs every tile: 2048 x 1024 x 32000 312 us instead of 293.)
    const bool few = MODE == kProducts && a.row.rows <= kFewRows;
    int few_target[2] = {-1, -1};
    float few_rest[2] = {0.f, 0.f};
    if (few) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = 32 * u + lane;
        if (r < a.row.rows) {
          const float4 f = *reinterpret_cast<const float4*>(a.info + r);
          few_target[u] = __float_as_int(f.w);
          few_rest[u] = lost(f.z);
        }
      }
    }
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* boxes = smem + Cfg::kOffBox + (warp - 2) * 2 * Cfg::kBox;
    const uint32_t acce_leader = map_peer(smem_u32(acce), 0);
    int staged = 0;
    // what the epilogue knows of its row of a tile, read a tile ahead
    auto row_of = [&](const Item& t) {
      const int m = MODE == kFew ? t.n0 + half * 32 + lane : t.m0 + rank * 128 + q * 32 + lane;
      HeadRow info = {0.f, 0.f, 0.f, -1};
      if ((MODE == kStats || MODE == kFew) && m < a.row.rows) {
        float w;
        info.target = head_target(a.row, m, w, nullptr);
      }
      if ((MODE == kGrad ||
           (MODE == kProducts && (t.kind == kLogits || (t.kind == kDh && a.dh_out == kDhBf16)))) &&
          m < a.row.rows) {
        const float4 f = *reinterpret_cast<const float4*>(a.info + m);
        info = HeadRow{f.x, f.y, f.z, __float_as_int(f.w)};
      }
      return info;
    };
    Item ahead;
    bool more = walk.next(a, ahead);
    HeadRow info_ahead = more ? row_of(ahead) : HeadRow{0.f, 0.f, 0.f, -1};
    for (int i = 0; more; ++i) {
      it = ahead;
      const HeadRow info = info_ahead;
      more = walk.next(a, ahead);
      if (more) info_ahead = row_of(ahead);
      const int b = i & 1;
      const int mw = it.m0 + rank * 128 + q * 32, m = mw + lane;  // the warp's first row, the thread's
      const int cw = it.n0 + half * 128;                          // the warp's first column
      const bool grad = MODE == kGrad || (MODE == kProducts && it.kind == kLogits);
      const int width = MODE != kProducts ? a.cols : (grad ? a.g_cols : a.row.d);
      const int target = info.target - (MODE == kGrad ? a.v0 : (MODE == kProducts ? a.g_v0 : 0));
      const float rest = MODE == kProducts && !grad && info.target >= 0 ? lost(info.gt) : 0.f;
      unsigned hits[2] = {0, 0};  // rows whose target is among the warp's 32 rows of dE
      if (few && it.kind == kDe) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          hits[u] = __ballot_sync(0xffffffffu, static_cast<unsigned>(few_target[u] - (a.v0 + mw)) < 32u);
      }
      head_wait(&accf[b], (i >> 1) & 1, err, DERR_ACC_WAIT, abort);
      tc_fence_after();
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * kTile + half * (Cfg::kColumns / 2);
      auto drained = [&] {  // the accumulator is free again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed(acce_leader + static_cast<uint32_t>(b * sizeof(uint64_t)));
      };
      if constexpr (MODE == kFew) {
        // the thread has 32 rows of h at one column of the vocabulary, and wants it the other way round
        uint32_t ra[32];
        tmem_ld32(tb, ra);
        tmem_ld_wait32(ra);
        drained();
        float* box = reinterpret_cast<float*>(boxes);
#pragma unroll
        for (int j = 0; j < 32; ++j) box[j * 33 + lane] = __uint_as_float(ra[j]);
        __syncwarp();
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = box[lane * 33 + j];
        __syncwarp();
        const bool clip = a.row.clip > 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (clip) v[j] = limit(v[j], a.row.clip);
          if (mw + j >= a.row.vocab || mw + j == info.target) v[j] = -INFINITY;
        }
        float rho;
        const float sum = to_powers<32>(v, rho);
        const int r = it.n0 + half * 32 + lane;
        if (r < a.row.rows)
          a.parts[static_cast<int64_t>(r) * (8 * a.m_tiles) + (mw / 32)] = make_float2(rho, sum);
      } else {
        // many columns at once: a load's latency is some 500 clocks, and 32 columns after the
        // other they were two thirds of the epilogue
        constexpr int kWide = MODE == kStats ? 128 : 64;
#pragma unroll 1
        for (int c1 = 0; c1 < 128; c1 += kWide) {
          uint32_t ra[kWide];
#pragma unroll
          for (int c = 0; c < kWide / 32; ++c) tmem_ld32(tb + c1 + c * 32, ra + c * 32);
#pragma unroll
          for (int c = 0; c < kWide / 32; ++c) tmem_ld_wait32(ra + c * 32);
          if (c1 + kWide == 128) drained();
          const int c0 = cw + c1;  // the first of these columns
          float v[kWide];
#pragma unroll
          for (int j = 0; j < kWide; ++j) v[j] = __uint_as_float(ra[j]);
          const bool edge = c0 + kWide > width;
          const bool has_target = static_cast<unsigned>(target - c0) < static_cast<unsigned>(kWide);
          if (MODE == kStats) {
            float rho;
            const bool kept = it.n0 < a.keep;
            uint32_t cut[kWide / 32] = {};  // columns beyond the limit
            if (a.row.clip > 0.f) {
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j) {
                if (kept) cut[j >> 5] |= fabsf(v[j]) > a.row.clip ? 1u << (j & 31) : 0u;
                v[j] = limit(v[j], a.row.clip);
              }
            }
            if (edge) {
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j)
                if (c0 + j >= width) v[j] = -INFINITY;
            }
            if (__any_sync(0xffffffffu, has_target)) {
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j)
                if (c0 + j == target) v[j] = -INFINITY;
            }
            const float sum = to_powers<kWide>(v, rho);
            if (m < a.row.rows)
              a.parts[static_cast<int64_t>(m) * (2 * a.n_tiles) + (it.n0 / 128 + half)] = make_float2(rho, sum);
            if (!kept) continue;
            if (a.row.clip > 0.f) {
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j) v[j] = cut[j >> 5] >> (j & 31) & 1u ? 0.f : v[j];
            }
          }
          if (grad) {
            const f32x2 l2 = pack2(kLog2e, kLog2e), ref = pack2(-info.rho, -info.rho);
            const f32x2 sc = pack2(info.scale, info.scale);
            if (a.row.clip > 0.f) {  // columns beyond the limit: marked, so that they come out as 0
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j) v[j] = fabsf(v[j]) > a.row.clip ? -INFINITY : v[j];
            }
#pragma unroll
            for (int j = 0; j < kWide; j += 2) {
              float x, y;
              unpack2(fma2(pack2(v[j], v[j + 1]), l2, ref), x, y);
              unpack2(mul2(pack2(ex2_approx(x), ex2_approx(y)), sc), v[j], v[j + 1]);
            }
            if (__any_sync(0xffffffffu, has_target)) {
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j)
                if (c0 + j == target) v[j] = info.gt;
            }
            if (__any_sync(0xffffffffu, info.target < 0)) {  // zeros, whatever the row holds
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j) v[j] = info.target < 0 ? 0.f : v[j];
            }
          }
          if (MODE == kProducts && !grad) {
            if (__any_sync(0xffffffffu, rest != 0.f)) {  // what g_t lost to its rounding
              __syncwarp();
              const __nv_bfloat16* e = a.emb + static_cast<int64_t>(max(info.target, 0)) * a.row.d + c0;
#pragma unroll
              for (int j = 0; j < kWide; j += 8) {
                if (c0 + j < width) {
                  float w[8];
                  load8(e + j, w);
#pragma unroll
                  for (int k = 0; k < 8; ++k) v[j + k] = fmaf(rest, w[k], v[j + k]);
                }
              }
            }
            if (hits[0] | hits[1]) {
#pragma unroll
              for (int u = 0; u < 2; ++u)
                for (unsigned todo = hits[u]; todo; todo &= todo - 1) {
                  const int l = __ffs(todo) - 1;
                  const int of = __shfl_sync(0xffffffffu, few_target[u], l) - (a.v0 + mw);
                  const float part = __shfl_sync(0xffffffffu, few_rest[u], l);
                  if (lane == of) {
                    const __nv_bfloat16* x = a.hm + (32 * u + l) * a.ldm + c0;
#pragma unroll
                    for (int j = 0; j < kWide; j += 8) {
                      if (c0 + j < width) {
                        float w[8];
                        load8(x + j, w);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[j + k] = fmaf(part, w[k], v[j + k]);
                      }
                    }
                  }
                  __syncwarp();
                }
            }
            const float al = it.kind == kDe || a.dh_out == kDhBf16 ? a.row.inv_count : 1.f;
#pragma unroll
            for (int j = 0; j < kWide; ++j) v[j] *= al;
            // rows that count for nothing: zeros, where a table with a NaN made 0 times it
            const bool none = it.kind == kDh && a.dh_out == kDhBf16 && info.target < 0;
            if (__any_sync(0xffffffffu, none)) {
              __syncwarp();
#pragma unroll
              for (int j = 0; j < kWide; ++j) v[j] = none ? 0.f : v[j];
            }
          }
          // out, 32 columns at a time, through the warp's two boxes
          const bool f32 = MODE == kProducts && !grad && (it.kind == kDe ? a.de_f32 : a.dh_out != kDhBf16);
#pragma unroll
          for (int c = 0; c < kWide / 32; ++c) {
            const int col = c0 + c * 32;
            if (col >= width) break;
            uint8_t* box = boxes + (staged++ & 1) * Cfg::kBox;
            if (lane == 0) wait_read_1();
            __syncwarp();
            const float* o = v + c * 32;
            if (f32) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                *reinterpret_cast<float4*>(box + box_f32(lane, u)) =
                    make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            } else if (MODE == kStats) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(box + box_bf16(lane, u)) =
                    make_uint4(pack_f16x2(o[8 * u], o[8 * u + 1]), pack_f16x2(o[8 * u + 2], o[8 * u + 3]),
                               pack_f16x2(o[8 * u + 4], o[8 * u + 5]), pack_f16x2(o[8 * u + 6], o[8 * u + 7]));
            } else {
#pragma unroll
              for (int u = 0; u < 4; ++u) store8(reinterpret_cast<__nv_bfloat16*>(box + box_bf16(lane, u)), o + 8 * u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (!*abort) {
                if (MODE != kProducts) {
                  tma_store_2d(&maps.c, col, mw, box);
                } else if (grad) {
                  tma_store_2d(&maps.c3, col, mw, box);
                } else if (it.kind == kDe) {
                  if (a.de_f32) tma_reduce_add_2d(&maps.c2, col, a.v0 + mw, box);
                  else tma_store_2d(&maps.c2, col, a.v0 + mw, box);
                } else {
                  const int y = it.split * a.rows_pad + mw;
                  if (a.dh_out == kDhAdd) tma_reduce_add_2d(&maps.c, col, y, box);
                  else tma_store_2d(&maps.c, col, y, box);
                }
              }
              bulk_commit();
            }
          }
        }
      }
    }
    griddep_launch();
    if (lane == 0) bulk_wait_read_all();
  }
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the pair's products may read its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// h with the rows that count for nothing set to zero, in rows that start on 128 bytes; a
// warp a row.
__global__ void __launch_bounds__(256) head_copy_kernel(HeadArgs a, const __nv_bfloat16* __restrict__ h, int64_t ldh,
                                                        __nv_bfloat16* __restrict__ hm, int64_t ldm) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.rows) return;
  float w;
  const bool live = head_target(a, r, w, nullptr) >= 0;
#pragma unroll 4
  for (int c = lane * 8; c < a.d; c += 256)
    *reinterpret_cast<uint4*>(hm + r * ldm + c) =
        live ? *reinterpret_cast<const uint4*>(h + r * ldh + c) : make_uint4(0, 0, 0, 0);
}

// W warps per row: they join the row's sums, take the target's logit as a dot product, the
// loss, what the gradient pass needs, and (hm not NULL) h with the rows that count for
// nothing set to zero.
template <int W>
__global__ void __launch_bounds__(256) head_rows_kernel(HeadArgs a, const __nv_bfloat16* __restrict__ h, int64_t ldh,
                                                        const __nv_bfloat16* __restrict__ emb,
                                                        const float2* __restrict__ parts, int nparts,
                                                        float* __restrict__ loss, HeadRow* __restrict__ info,
                                                        __nv_bfloat16* __restrict__ hm, int64_t ldm, int* err) {
  static_assert(W == 1 || W == 8, "a warp or the CTA");
  griddep_launch();
  __shared__ float shared[3][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = W == 1 ? blockIdx.x * 8 + warp : blockIdx.x;
  const int at = W == 1 ? lane : threadIdx.x;
  if (r >= a.rows) {
    griddep_wait();
    return;
  }
  // before the wait: the call's inputs and hm, which its other launches do not touch before
  // this one has ended (launched by the stats kernel, which had waited itself)
  float w;
  const int t = head_target(a, r, w, at == 0 ? err : nullptr);
  float zt = 0.f;
  for (int c = at * 8; c < a.d; c += 256 * W) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (t >= 0) {
      u = *reinterpret_cast<const uint4*>(h + r * ldh + c);
      float e[8];
      load8(emb + static_cast<int64_t>(t) * a.d + c, e);
      const float2 p0 = unpack_bf16x2(u.x), p1 = unpack_bf16x2(u.y), p2 = unpack_bf16x2(u.z), p3 = unpack_bf16x2(u.w);
      zt += ((p0.x * e[0] + p0.y * e[1]) + (p1.x * e[2] + p1.y * e[3])) +
            ((p2.x * e[4] + p2.y * e[5]) + (p3.x * e[6] + p3.y * e[7]));
    }
    if (hm) *reinterpret_cast<uint4*>(hm + r * ldm + c) = u;
  }
  zt = warp_sum(zt);
  griddep_wait();
  if (t < 0) {
    if (at == 0) {
      loss[r] = 0.f;
      if (info) info[r] = HeadRow{0.f, 0.f, 0.f, -1};
    }
    return;
  }
  const float2* mine = parts + static_cast<int64_t>(r) * nparts;
  float rho = -INFINITY, s = 0.f;
#pragma unroll 4
  for (int i = at; i < nparts; i += 32 * W) {
    const float2 p = mine[i];
    const float to = fmaxf(rho, p.x);
    if (to > -INFINITY) s = s * exp2f(rho - to) + p.y * exp2f(p.x - to);
    else s += p.y;  // nothing there, or NaN
    rho = to;
  }
  auto join = [&](float rx, float x, float ry, float y) {
    const float to = fmaxf(rx, ry);
    s = to > -INFINITY ? x * exp2f(rx - to) + y * exp2f(ry - to) : x + y;
    rho = to;
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float rho2 = __shfl_xor_sync(0xffffffffu, rho, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    if (lane & o) join(rho2, s2, rho, s);  // (in a fixed order for both lanes of a pair, so that all agree)
    else join(rho, s, rho2, s2);
  }
  if (W > 1) {
    if (lane == 0) {
      shared[0][warp] = rho;
      shared[1][warp] = s;
      shared[2][warp] = zt;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < W; ++i) {
      join(rho, s, shared[0][i], shared[1][i]);
      zt += shared[2][i];
    }
  }
  if (lane != 0) return;
  bool cut = false;
  if (a.clip > 0.f) {
    cut = fabsf(zt) > a.clip;
    zt = limit(zt, a.clip);
  }
  // odds of all other tokens together against the target: s 2^x.  (A logit of +inf makes the others' s
  // NaN by inf - inf; the target's is not among them)
  const float x = zt == INFINITY ? NAN : fmaf(-zt, kLog2e, rho);
  const float odds = s * exp2f(x);
  const float nll = x > 60.f ? fmaf(x, kLn2, logf(s)) : log1pf(odds);
  loss[r] = w * a.inv_count * nll;
  if (!info) return;
  const float ref = fmaxf(rho, ceilf(zt * kLog2e));
  const float total = (rho > -INFINITY ? s * exp2f(rho - ref) : s) + exp2f(fmaf(zt, kLog2e, -ref));
  // x > 60: the others have all of it
  const float others = x > 60.f ? (s == s ? 1.f : s) : odds / (1.f + odds);
  info[r] = HeadRow{ref, w / total, cut ? 0.f : -w * others, t};
}

// g of the first piece from the powers that the first pass left in its place: 16 elements
// a thread, all of one reference.
__global__ void __launch_bounds__(256) head_scale_kernel(int cols, int64_t ldg, int slabs,
                                                         const HeadRow* __restrict__ info,
                                                         const float2* __restrict__ parts, int nparts, uint4* g) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x / slabs, c = (blockIdx.x % slabs * 256 + threadIdx.x) * 16;
  if (c >= cols) return;
  const float4 f = *reinterpret_cast<const float4*>(info + r);
  const int target = __float_as_int(f.w);
  const float ref = parts[static_cast<int64_t>(r) * nparts + c / 128].x;
  uint4* at = g + (r * ldg + c) / 8;
  uint4 u[2] = {at[0], at[1]};
  // (a reference of -inf: powers of 0)
  const float k = ref == -INFINITY ? 0.f : f.y * exp2f(ref - f.x);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 p = unpack_f16x2(w[j]);
      p.x *= k;
      p.y *= k;
      const int col = c + 8 * i + 2 * j;
      if (col == target) p.x = f.z;
      if (col + 1 == target) p.y = f.z;
      w[j] = target < 0 ? 0u : pack_bf16x2(p.x, p.y);  // no target: zeros, whatever the row holds
    }
    at[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// dh = inv_count times the sum of its parts and of what g_t lost to its rounding, 8 columns
// a thread (a warp a row waits 11 us for 16 parts of 64 rows).
__global__ void __launch_bounds__(256) head_dh_kernel(int rows, int d, int splits, int rows_pad, float scale,
                                                      const float* __restrict__ src, const HeadRow* __restrict__ info,
                                                      const __nv_bfloat16* __restrict__ emb,
                                                      __nv_bfloat16* __restrict__ dh, int64_t lddh) {
  griddep_wait();
  griddep_launch();
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;
  const uint32_t groups = d / 8;
  const int r = static_cast<int>(i / groups), c = static_cast<int>(i % groups) * 8;
  if (r >= rows) return;
  const float4 f = *reinterpret_cast<const float4*>(info + r);
  const int target = __float_as_int(f.w);
  const float rest = target >= 0 ? lost(f.z) : 0.f;
  float v[8], u[8];
  load8(emb + static_cast<int64_t>(max(target, 0)) * d + c, u);
  const float* at = src + static_cast<int64_t>(r) * d + c;
  load8(at, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fmaf(rest, u[j], v[j]);
#pragma unroll 8
  for (int p = 1; p < splits; ++p) {
    load8(at + static_cast<int64_t>(p) * rows_pad * d, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += u[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = target < 0 ? 0.f : v[j] * scale;  // (0 times a table with a NaN is none)
  store8(dh + r * lddh + c, v);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
int check(const char* what) {
  count_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(GPIPE_ERR_CUDA, "head_loss: %s launch: %s", what, cudaGetErrorString(e));
  return GPIPE_OK;
}

int up_to(int n, int m) { return (n + m - 1) / m; }

bool sizes_ok(int rows, int d, int vocab, int piece) {
  return rows >= 1 && rows <= (1 << 24) && d >= 8 && d <= (1 << 16) && d % 8 == 0 && vocab >= 1 &&
         vocab <= (1 << 27) && piece >= 0 &&
         static_cast<int64_t>(up_to(rows, kTile)) * up_to(vocab, kTile) <= (1 << 26);
}

// Columns of a piece: a multiple of 256; 0 asks for as many as make g 256 MB, in one piece or
// in two at a time.
int piece_columns(int rows, int vocab, int piece) {
  int64_t p = piece ? piece : std::max<int64_t>(2048, (static_cast<int64_t>(1) << 27) / rows);
  if (!piece && p < vocab) p = std::max<int64_t>(2048, p / 2);
  p = std::min<int64_t>((p + kTile - 1) / kTile * kTile, (static_cast<int64_t>(vocab) + kTile - 1) / kTile * kTile);
  return static_cast<int>(p);
}

// How the pairs share dE's and g's tiles, and about how many k-blocks the busiest has.  A
// tile costs its k-blocks and two more (measured: filling the ring and the last tile's
// epilogue).
struct Plan {
  Share de, g;
  int64_t longest;
};
Plan plan(int64_t dh_items, int dh_nk, int64_t de_items, int de_nk, int64_t g_items, int g_nk, int pairs) {
  const int64_t ch = dh_nk + 2, ce = de_nk + 2, cg = g_nk + 2, q = dh_items / pairs, late = dh_items % pairs,
                rest = pairs - late;
  const int64_t ahead = late ? std::min((ch + ce / 2) / ce, de_items / rest) : 0, left = de_items - ahead * rest;
  // what the pairs with one tile of dh less still have in hand, or those with one of dE less
  const int64_t gap = late ? ch - ahead * ce : 0, late2 = gap > ce ? late : left % pairs,
                gap2 = gap > ce ? gap : (late2 ? ce : 0);
  const int64_t ahead2 = late2 ? std::min((gap2 + cg / 2) / cg, g_items / (pairs - late2)) : 0;
  const int64_t before = q * ch + std::max<int64_t>(late ? ch : 0, ahead * ce) + (left + pairs - 1) / pairs * ce;
  const int64_t even = (dh_items * ch + de_items * ce + g_items * cg + pairs - 1) / pairs + cg;
  return {{static_cast<int>(de_items), static_cast<int>(late), static_cast<int>(ahead)},
          {static_cast<int>(g_items), static_cast<int>(late2), static_cast<int>(ahead2)},
          g_items ? std::max(before, even) : before};
}

// Parts of dh's K (the vocabulary): with few tiles of dh their long sums would be what
// all else waits for.  Depends on the sizes and on whether dE is wanted, as do then the bits
// of dh.
int dh_splits(int rows, int d, int cols, bool demb, bool more) {
  const int64_t tiles = static_cast<int64_t>(up_to(rows, kTile)) * up_to(d, kTile);
  const int64_t de_items = demb ? static_cast<int64_t>(up_to(cols, kTile)) * up_to(d, kTile) : 0;
  const int64_t g_items = more ? static_cast<int64_t>(up_to(rows, kTile)) * up_to(cols, kTile) : 0;
  const int nk = up_to(cols, kK), de_nk = up_to(rows, kK);
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= 64 && nk / s >= 8; ++s) {
    // a part's 8 bytes an element through memory: 4 k-blocks' time a tile; the last kernel
    // reads eight parts at a time, in about 2
    const int64_t cost = plan(tiles * s, up_to(nk, s), de_items, de_nk, g_items, up_to(d, kK), kPlanPairs).longest +
                         (s > 1 ? 8 + 4 * s * tiles / kPlanPairs + s / 4 : 0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

struct HeadScratch {
  size_t parts, info, hm, g, g2, dh, bytes;
  int cols, splits, rows_pad, ldm;
  bool direct;  // dh comes out of the products as it is
  bool keep;    // the first piece's powers are kept
  bool copy;    // the products read a copy of h
};
HeadScratch head_scratch(int rows, int d, int vocab, int piece, int grads, bool apart) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  const size_t n = static_cast<size_t>(rows);
  HeadScratch s;
  s.cols = piece_columns(rows, vocab, piece);
  s.splits = grads & 1 ? dh_splits(rows, d, s.cols, grads & 2, s.cols < vocab) : 1;
  s.rows_pad = up_to(rows, kTile) * kTile;
  s.direct = s.splits == 1 && s.cols >= vocab;
  // (a tile is made again for 256 rows, however few there are)
  s.keep = grads && static_cast<int64_t>(d) * s.rows_pad >= static_cast<int64_t>(kKeepWidth) * rows;
  s.ldm = up_to(d, kK) * kK;  // copies of rows that start on 128 bytes: d = 712 is 20 % slower than 704 or 720
  s.parts = 0;
  s.info = up(n * (!grads && rows <= kFewRows ? 8 : 2) * up_to(vocab, kTile) * sizeof(float2));
  s.hm = s.info + (grads ? up(n * sizeof(HeadRow)) : 0);
  s.copy = apart && rows > kFewRows && static_cast<int64_t>(rows) * vocab >= kCopyWork / d;
  s.g = s.hm + (s.copy || (grads & 2) ? up(n * s.ldm * 2) : 0);
  s.g2 = s.g + (grads ? up(n * s.cols * 2) : 0);
  s.dh = s.g2 + (grads && s.cols < vocab ? up(n * s.cols * 2) : 0);
  s.bytes = s.dh + ((grads & 1) && !s.direct ? up(static_cast<size_t>(s.splits) * s.rows_pad * d * 4) : 0);
  return s;
}

// 2-D tensor of `outer` rows of `inner` elements, ld elements apart; boxes of
// box_inner x box_outer.  Boxes that leave (32 x 32) have rows of 64 bytes in bf16.
bool head_map(CUtensorMap* m, const void* base, bool f32, int64_t inner, int64_t outer, int64_t ld, int box_inner,
              int box_outer) {
  using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn enc = known.load(std::memory_order_acquire);
  if (!enc) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    enc = reinterpret_cast<EncodeFn>(p);
    known.store(enc, std::memory_order_release);
  }
  const int es = f32 ? 4 : 2;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  cuuint32_t estr[2] = {1u, 1u};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_inner * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// early: launched while the launch before it runs, as only one behind another of the call is.
// A CTA has most of an SM's shared memory and all of its tensor memory, and one that waited for a
// foreign kernel would keep them from other streams for as long as that takes (a product of 0.7 ms
// beside a call that waited for 25 ms of one CTA took those 25); within the call it is the launch
// before's last tile or some microseconds.  The first pass gives some of its start away by that:
// calls in a row 18.6 us for 16.5 (5 x 64 x 517, both gradients), 22.6 for 19.1 (1 x 1024 x 32000),
// 294 for 291 (2048 x 1024 x 32000, both), 57 for 51 (1 x 1024 x 131072).
template <Mode MODE>
int launch_head_gemm(const HeadMaps& maps, const HeadGemm& a, int64_t items, bool early, int* err, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const int rc = once_per_device(done, [] {
    const cudaError_t e = cudaFuncSetAttribute(head_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               HeadCfg<MODE>::kSmem);
    return e == cudaSuccess ? GPIPE_OK
                            : set_error(GPIPE_ERR_CUDA, "head_loss: smem attribute: %s", cudaGetErrorString(e));
  });
  if (rc) return rc;
  const int pairs = static_cast<int>(std::min<int64_t>(std::max(1, num_sms() / 2), items));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kHeadThreads);
  cfg.dynamicSmemBytes = HeadCfg<MODE>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  set_priority_attr(attr[1], s);
  attr[2].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[2].val.programmaticStreamSerializationAllowed = early && pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 3;
  HeadGemm b = a;
  if (MODE == kProducts) {
    const Plan p = plan(a.dh_items, up_to(up_to(a.cols, kK), a.splits), a.de.n, up_to(a.row.rows, kK), a.g.n,
                        up_to(a.row.d, kK), pairs);
    b.de = p.de;
    b.g = p.g;
  }
  (void)cudaLaunchKernelEx(&cfg, head_gemm_kernel<MODE>, maps, b, err);
  return check(MODE == kStats || MODE == kFew ? "stats" : (MODE == kGrad ? "gradient" : "products"));
}

}  // namespace

size_t head_loss_scratch_bytes(int rows, int d, int vocab, int piece, int grads) {
  if (!sizes_ok(rows, d, vocab, piece) || grads < 0 || grads > 3) return 0;
  return head_scratch(rows, d, vocab, piece, grads, true).bytes;  // (h may lie in any way)
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
                     "head_loss: need 1 <= rows <= 2^24, 8 <= d <= 2^16, d %% 8 == 0, 1 <= vocab <= 2^27, "
                     "piece >= 0 and at most 2^26 tiles of 256 x 256");
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
  const bool apart = (reinterpret_cast<uintptr_t>(h) | static_cast<uintptr_t>(ldh) * 2) % 32 != 0;
  const HeadScratch at = head_scratch(rows, d, vocab, piece, grads, apart);
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
  auto* parts = reinterpret_cast<float2*>(w + at.parts);
  auto* info = reinterpret_cast<HeadRow*>(w + at.info);
  auto* hm = reinterpret_cast<__nv_bfloat16*>(w + at.hm);
  auto* g = reinterpret_cast<__nv_bfloat16*>(w + at.g);
  float* dh32 = reinterpret_cast<float*>(w + at.dh);
  const auto* e = static_cast<const __nv_bfloat16*>(emb);
  const HeadArgs a{rows, d, vocab, seq, row0, tokens, row_weight, inv_count, clip};
  HeadMaps maps = {};
  HeadGemm q = {};
  q.row = a;
  q.cols = vocab;
  q.m_tiles = up_to(rows, kTile);
  q.n_tiles = up_to(vocab, kTile);
  q.parts = parts;
  q.info = info;
  q.emb = e;
  q.hm = hm;
  q.ldm = at.ldm;
  const bool few = !grads && rows <= kFewRows;
  const int nparts = (few ? 8 : 2) * q.n_tiles;
  CUtensorMap map_h;
  int rc;
  if (at.copy) {
    (void)launch_k(head_copy_kernel, up_to(rows, 8), 256, 0, st, a, static_cast<const __nv_bfloat16*>(h), ldh, hm,
                   static_cast<int64_t>(at.ldm));
    if ((rc = check("copy"))) return rc;
  }
  // (kFew has h as the other operand, in boxes of its own; it is never copied)
  bool ok = head_map(&map_h, at.copy ? hm : h, false, d, rows, at.copy ? at.ldm : ldh, kK, few ? kFewRows / 2 : 128) &&
            head_map(&maps.b, emb, false, d, vocab, d, kK, 128);
  if (ok && at.keep) {
    q.keep = at.cols;
    ok = head_map(&maps.c, g, false, std::min(at.cols, vocab), rows, at.cols, 32, 32);
  }
  if (!ok) return set_error(GPIPE_ERR_CUDA, "head_loss: cuTensorMapEncodeTiled failed");
  maps.a = map_h;
  if (few) {  // the vocabulary as rows
    std::swap(maps.a, maps.b);
    std::swap(q.m_tiles, q.n_tiles);
    rc = launch_head_gemm<kFew>(maps, q, q.m_tiles, false, err, st);
  } else {
    rc = launch_head_gemm<kStats>(maps, q, static_cast<int64_t>(q.m_tiles) * q.n_tiles, at.copy, err, st);
  }
  if (rc) return rc;
  const auto* hb = static_cast<const __nv_bfloat16*>(h);
  const float2* in_parts = parts;
  HeadRow* rows_info = grads ? info : nullptr;
  __nv_bfloat16* to_copy = demb && !at.copy ? hm : nullptr;
  // with few rows a warp each would take long over their sums: 3 rows over 128616 columns 14 us
  if (rows <= kWideRows && nparts >= 128)
    (void)launch_k(head_rows_kernel<8>, rows, 256, 0, st, a, hb, ldh, e, in_parts, nparts, loss_rows, rows_info,
                   to_copy, static_cast<int64_t>(at.ldm), err);
  else
    (void)launch_k(head_rows_kernel<1>, up_to(rows, 8), 256, 0, st, a, hb, ldh, e, in_parts, nparts, loss_rows,
                   rows_info, to_copy, static_cast<int64_t>(at.ldm), err);
  if ((rc = check("rows"))) return rc;
  __nv_bfloat16* now = g;
  __nv_bfloat16* then = reinterpret_cast<__nv_bfloat16*>(w + at.g2);
  q.n_tiles = up_to(std::min(at.cols, vocab), kTile);
  if (grads) {
    const int cols = std::min(at.cols, vocab);
    if (at.keep) {
      const int slabs = up_to(cols, 16 * 256);
      (void)launch_k(head_scale_kernel, rows * slabs, 256, 0, st, cols, static_cast<int64_t>(at.cols), slabs,
                     static_cast<const HeadRow*>(info), in_parts, nparts, reinterpret_cast<uint4*>(g));
      if ((rc = check("scale"))) return rc;
    } else {
      q.cols = cols;
      ok = (cols == vocab || head_map(&maps.b, emb, false, d, cols, d, kK, 128)) &&
           head_map(&maps.c, g, false, cols, rows, at.cols, 32, 32);
      if (!ok) return set_error(GPIPE_ERR_CUDA, "head_loss: cuTensorMapEncodeTiled failed");
      rc = launch_head_gemm<kGrad>(maps, q, static_cast<int64_t>(q.m_tiles) * q.n_tiles, true, err, st);
      if (rc) return rc;
    }
  }
  for (int v0 = 0; grads && v0 < vocab; v0 += at.cols, std::swap(now, then)) {
    const int cols = std::min(at.cols, vocab - v0), next = v0 + cols;
    const auto* piece_of_e = e + static_cast<int64_t>(v0) * d;
    q.cols = cols;
    q.v0 = v0;
    q.g_v0 = next;
    q.g_cols = std::min(at.cols, vocab - next);
    q.g_tiles = up_to(q.g_cols, kTile);
    q.g.n = q.m_tiles * q.g_tiles;
    ok = true;
    if (q.g.n) {
      maps.a3 = map_h;
      ok = head_map(&maps.b3, e + static_cast<int64_t>(next) * d, false, d, q.g_cols, d, kK, 128) &&
           head_map(&maps.c3, then, false, q.g_cols, rows, at.cols, 32, 32);
    }
    q.n_tiles = up_to(d, kTile);
    q.splits = std::min(at.splits, up_to(cols, kK));
    q.rows_pad = at.rows_pad;
    q.dh_items = dh ? q.m_tiles * q.n_tiles * q.splits : 0;
    q.de.n = demb ? up_to(cols, kTile) * q.n_tiles : 0;
    q.dh_out = at.direct ? kDhBf16 : (v0 ? kDhAdd : kDhStore);
    q.de_f32 = demb_dtype == DT_F32;
    if (ok && dh) {
      ok = head_map(&maps.a, now, false, cols, rows, at.cols, kK, 128) &&
           head_map(&maps.b, piece_of_e, false, d, cols, d, kK, kK) &&
           (at.direct ? head_map(&maps.c, dh, false, d, rows, lddh, 32, 32)
                      : head_map(&maps.c, dh32, true, d, static_cast<int64_t>(at.splits) * at.rows_pad, d, 32, 32));
    }
    if (ok && demb)
      ok = head_map(&maps.a2, now, false, cols, rows, at.cols, kK, kK) &&
           head_map(&maps.b2, hm, false, d, rows, at.ldm, kK, kK) &&
           head_map(&maps.c2, demb, q.de_f32, d, vocab, d, 32, 32);
    if (!ok) return set_error(GPIPE_ERR_CUDA, "head_loss: cuTensorMapEncodeTiled failed");
    const int64_t items = static_cast<int64_t>(q.dh_items) + q.de.n + q.g.n;
    if ((rc = launch_head_gemm<kProducts>(maps, q, items, true, err, st))) return rc;
  }
  if (!dh || at.direct) return GPIPE_OK;
  const auto ctas = static_cast<unsigned>((static_cast<int64_t>(rows) * (d / 8) + 255) / 256);
  (void)launch_k(head_dh_kernel, ctas, 256, 0, st, rows, d, at.splits, at.rows_pad, inv_count,
                 static_cast<const float*>(dh32), static_cast<const HeadRow*>(info), e, static_cast<__nv_bfloat16*>(dh),
                 lddh);
  return check("dh");
}

}  // namespace gp
