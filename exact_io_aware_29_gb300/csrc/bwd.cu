// Backward pass of the fixed and packed layouts (the kernels of bwd_kernel.cuh
// compiled for them) and the fixed scratch of the allocation-free entry point.
#include <mutex>

#include <cudaTypedefs.h>

#include "bwd_kernel.cuh"

namespace fa {

// ---------------------------------------------------------------------------
// Fixed scratch for the allocation-free backward entry point. Some callers
// cannot call cudaMalloc (or any allocating routine) at the point where they
// need the backward, e.g. code running inside a memory pool or allocator
// hook, or a host framework whose device memory is owned by another
// subsystem. For them the backward workspace lives in this static device
// array instead: every GPU that loads the library reserves it until the
// process exits. In host code the array's name is only a host-side stand-in;
// its device address comes from cudaGetSymbolAddress, once per device (and
// again if the device's context was torn down and recreated, e.g. after
// cudaDeviceReset: the module is then loaded anew and the array may move).
// ---------------------------------------------------------------------------
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

// Unique id of the calling thread's current context (0 if the driver cannot
// tell), through the driver entry points the runtime exposes.
static unsigned long long current_context_id() {
  static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
  });
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (get_current == nullptr || get_id == nullptr || get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr ||
      get_id(ctx, &id) != CUDA_SUCCESS)
    return 0;
  return id;
}

cudaError_t noalloc_scratch(void** ptr, size_t* bytes) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static void* addr[kMaxDevices] = {};
  static unsigned long long ctx_of[kMaxDevices] = {};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  e = cudaSetDevice(dev);  // binds (and if needed creates) the device's primary context
  if (e != cudaSuccess) return e;
  const unsigned long long ctx = current_context_id();
  std::lock_guard<std::mutex> lk(mu);
  if (addr[dev] == nullptr || ctx_of[dev] != ctx) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);  // with `dev` current
    if (e != cudaSuccess) return e;
    addr[dev] = p;
    ctx_of[dev] = ctx;
  }
  *ptr = addr[dev];
  *bytes = kNoAllocScratchBytes;
  return cudaSuccess;
}

cudaError_t set_bwd_test_hooks(unsigned long long wait_limit_ns, int drop_loads, cudaStream_t stream) {
  return set_test_hooks_here(wait_limit_ns, drop_loads, stream);
}

int take_bwd_status() { return take_status_here(); }

cudaError_t launch_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                       const BwdArgs& a, cudaStream_t stream, const LaunchMarks* m) {
  const bool c = a.s.causal != 0;
  if (a.pk.varlen) {
    if (a.s.D == 64)
      return c ? launch_bwd_order<64, true, kPacked>(tq, tk, tv, tdo, a, stream, m)
               : launch_bwd_order<64, false, kPacked>(tq, tk, tv, tdo, a, stream, m);
    return c ? launch_bwd_order<128, true, kPacked>(tq, tk, tv, tdo, a, stream, m)
             : launch_bwd_order<128, false, kPacked>(tq, tk, tv, tdo, a, stream, m);
  }
  if (a.s.D == 64)
    return c ? launch_bwd_order<64, true, kFixed>(tq, tk, tv, tdo, a, stream, m)
             : launch_bwd_order<64, false, kFixed>(tq, tk, tv, tdo, a, stream, m);
  return c ? launch_bwd_order<128, true, kFixed>(tq, tk, tv, tdo, a, stream, m)
           : launch_bwd_order<128, false, kFixed>(tq, tk, tv, tdo, a, stream, m);
}

}  // namespace fa
