// Backward of prompt attention with grouped heads: the backward kernels
// compiled for the grouped packed layout. A work item is (sequence, key head,
// 128-key block) and loops over the query blocks of all G query heads of the
// key head, so dK and dV are summed over the group in the TMEM accumulators:
// no atomics, no second pass over per-head gradients, and K_j and V_j are
// loaded once for G heads.
#include "bwd_kernel.cuh"

namespace fa {

cudaError_t set_bwd_gqa_test_hooks(unsigned long long wait_limit_ns, int drop_loads, cudaStream_t stream) {
  return set_test_hooks_here(wait_limit_ns, drop_loads, stream);
}

int take_bwd_gqa_status() { return take_status_here(); }

cudaError_t launch_bwd_gqa(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t stream, const LaunchMarks* m) {
  const bool c = a.s.causal != 0;
  if (a.s.D == 64)
    return c ? launch_bwd_order<64, true, kGrouped>(tq, tk, tv, tdo, a, stream, m)
             : launch_bwd_order<64, false, kGrouped>(tq, tk, tv, tdo, a, stream, m);
  return c ? launch_bwd_order<128, true, kGrouped>(tq, tk, tv, tdo, a, stream, m)
           : launch_bwd_order<128, false, kGrouped>(tq, tk, tv, tdo, a, stream, m);
}

}  // namespace fa
