// Forward pass of the fixed and packed layouts: the kernels of fwd_kernel.cuh
// compiled for them.
#include "fwd_kernel.cuh"

namespace fa {

cudaError_t set_fwd_test_hooks(unsigned long long wait_limit_ns, int drop_loads, cudaStream_t stream) {
  return set_test_hooks_here(wait_limit_ns, drop_loads, stream);
}

int take_fwd_status() { return take_status_here(); }

cudaError_t launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FwdArgs& a,
                       cudaStream_t stream, const LaunchMarks* m) {
  const bool c = a.s.causal != 0;
  if (a.pk.varlen) {
    if (a.s.D == 64)
      return c ? launch_fwd_t<64, true, kPacked>(tq, tk, tv, a, stream, m)
               : launch_fwd_t<64, false, kPacked>(tq, tk, tv, a, stream, m);
    return c ? launch_fwd_t<128, true, kPacked>(tq, tk, tv, a, stream, m)
             : launch_fwd_t<128, false, kPacked>(tq, tk, tv, a, stream, m);
  }
  if (a.s.D == 64)
    return c ? launch_fwd_t<64, true, kFixed>(tq, tk, tv, a, stream, m)
             : launch_fwd_t<64, false, kFixed>(tq, tk, tv, a, stream, m);
  return c ? launch_fwd_t<128, true, kFixed>(tq, tk, tv, a, stream, m)
           : launch_fwd_t<128, false, kFixed>(tq, tk, tv, a, stream, m);
}

}  // namespace fa
