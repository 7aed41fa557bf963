// Kernel launch with programmatic dependent launch (PDL).
//
// Kernels of the library start with griddep_wait() before they touch
// global memory (two named below aside), which blocks until the preceding kernel in the stream has
// completed and its writes are visible; so letting the next kernel launch
// early (PDL) only overlaps its launch and prologue with the predecessor's
// tail, and never changes a result.  Kernels call griddep_launch() once their
// remaining work no longer needs the SM resources a waiting successor would
// take.
//
// Two kernels of the head's loss touch global memory before their wait: the one that joins
// a row's sums reads the call's inputs and writes the copy of h, and the one that makes the
// gradient reads h (or its copy) and the table.  Both stand behind that call's first pass over
// the logits, which lets its successor launch only after its own griddep_wait(): whatever
// came before the call has completed then, and no launch of the call between that pass and
// them writes what they read or reads what they write.  This holds as long as the pass
// waits before it lets go and no kernel that breaks it is put between them.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <utility>

namespace gp {

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Whether launches made by this thread may overlap their predecessor (set by
// the step executor; default on).
bool pdl_enabled();
void set_pdl_enabled(bool on);

// heavy = true: the kernel holds most of an SM's shared memory / tensor
// memory and is not launched early, so that a waiting copy cannot keep those from
// kernels of other streams.  (One that takes its tensor memory after griddep_wait()
// and whose predecessor lets it launch only at its very end, when nothing but stores
// is left, may still go without: the windowed attention's backward kernel.  So may one
// whose predecessor is of the same call and as short as its own launch, or fills the SMs itself:
// the head loss's products behind its first pass, which is not launched early itself unless
// the call copies h first.)
// Every launch carries its stream's priority as a launch attribute, so that a
// kernel captured into a graph (instantiated with node priorities) keeps the
// priority of the stream it was issued to: the step's critical-path streams
// get SMs before its weight-gradient streams.
inline void set_priority_attr(cudaLaunchAttribute& a, cudaStream_t s) {
  int prio = 0;
  if (cudaStreamGetPriority(s, &prio) != cudaSuccess) prio = 0;
  a.id = cudaLaunchAttributePriority;
  a.val.priority = prio;
}

template <bool heavy = false, typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = (!heavy && pdl_enabled()) ? 1 : 0;
  set_priority_attr(attr[1], s);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Run f (a per-device setup such as a kernel attribute, which CUDA keeps per
// device) once for each device it succeeds on; devices >= 64 run it every time.
template <typename F>
int once_per_device(std::atomic<unsigned long long>& done, F&& f) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return f();
  const unsigned long long bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return 0;
  const int rc = f();
  if (rc == 0) done.fetch_or(bit, std::memory_order_acq_rel);
  return rc;
}

// Counts that the driver answers (above 0), by device and a small key, each asked
// for once.  A query that fails is not remembered, nor are the answers of devices >= 64.
template <int KEYS>
class PerDevice {
 public:
  template <typename F>  // cudaError_t(int*)
  cudaError_t get(int key, F&& ask, int* out) {
    int dev = 0;
    std::atomic<int>* at =
        cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 ? &kept_[dev][key] : nullptr;
    int n = at ? at->load(std::memory_order_relaxed) : 0;
    if (n < 1) {
      const cudaError_t e = ask(&n);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidValue;
      if (at) at->store(n, std::memory_order_relaxed);
    }
    *out = n;
    return cudaSuccess;
  }

 private:
  std::atomic<int> kept_[64][KEYS] = {};
};

}  // namespace gp
