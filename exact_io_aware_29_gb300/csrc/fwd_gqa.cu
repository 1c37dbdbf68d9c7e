// Prompt attention with grouped heads: the forward kernel compiled for the
// grouped packed layout (Hk key heads, G = H / Hk query heads each).
//
// A Q tile holds P heads of one group side by side (row = token * P + head; a
// TMA box of [128 / P tokens][P heads][64 columns] lands in that order), so a
// key block that is loaded once serves the P heads, and a short prompt fills
// its tiles: with G = 4, 64 tokens of four heads are the two tiles of one CTA
// instead of four CTAs with 64 of their 256 rows in use. For long prompts the
// number of tiles, of key blocks and of masked diagonal blocks stays the same,
// and the two tiles of a CTA, now only 2 * 128 / P tokens apart, visit equally
// many key blocks.
#include "fwd_kernel.cuh"

namespace fa {

cudaError_t set_fwd_gqa_test_hooks(unsigned long long wait_limit_ns, int drop_loads, cudaStream_t stream) {
  return set_test_hooks_here(wait_limit_ns, drop_loads, stream);
}

int take_fwd_gqa_status() { return take_status_here(); }

cudaError_t launch_fwd_gqa(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const FwdGroupedArgs& a, cudaStream_t stream, const LaunchMarks* m) {
  const bool c = a.s.causal != 0;
  if (a.s.D == 64)
    return c ? launch_fwd_t<64, true, kGrouped>(tq, tk, tv, a, stream, m)
             : launch_fwd_t<64, false, kGrouped>(tq, tk, tv, a, stream, m);
  return c ? launch_fwd_t<128, true, kGrouped>(tq, tk, tv, a, stream, m)
           : launch_fwd_t<128, false, kGrouped>(tq, tk, tv, a, stream, m);
}

}  // namespace fa
