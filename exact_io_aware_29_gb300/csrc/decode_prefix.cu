// The prefix part of a shared-prefix decoding step as a dense product: the
// forward kernel compiled for the shared-prefix layout. Its Q tiles hold the
// queries of the sequences behind one prefix (row = sequence * P + head), its
// K and V blocks come from the prefix's pages, two 64-token boxes each, and a
// CTA covers one range of the keys for up to 256 rows, so that the prefix is
// read once per 256 rows instead of once per sequence. Each row's partial O
// (fp32, normalised) and log-sum go to the step's workspace and are joined
// with the sequence's own part by the step's last kernel. P goes to the product
// with V as f16 (2^-11 of each term; the streamed parts' hi + lo bf16 would be
// two products on the pipe that bounds this one): 8 times finer than the
// output's own rounding.
#include "fwd_kernel.cuh"

namespace fa {

cudaError_t set_decode_prefix_test_hooks(unsigned long long wait_limit_ns, int drop_loads, cudaStream_t stream) {
  return set_test_hooks_here(wait_limit_ns, drop_loads, stream);
}

int take_decode_prefix_status() { return take_status_here(); }

template <int D>
static cudaError_t launch_prefix_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const SharedArgs& d, QTile qt, cudaStream_t stream, const LaunchMarks* marks) {
  using C = FwdCfg<D>;
  auto kern = fa_fwd_kernel<D, false, kShared>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  FwdSharedArgs a{};
  a.dec = d;
  a.qt = qt;
  a.s.B = d.B;
  a.s.H = d.H;
  a.s.Hk = d.Hk;
  a.s.D = d.D;
  a.s.scale_log2 = d.scale_log2;
  const long long blocks = static_cast<long long>(d.prefix_splits) * d.P * (d.H / qt.P) *
                           ((d.max_group + 2 * qt.tok - 1) / (2 * qt.tok));
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  mark(marks, true, 0, stream);
  kern<<<static_cast<unsigned>(blocks), C::THREADS, C::SMEM_BYTES, stream>>>(tq, tk, tv, a);
  mark(marks, false, 0, stream);
  return cudaGetLastError();
}

cudaError_t launch_decode_prefix(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const SharedArgs& a, QTile qt, cudaStream_t stream, const LaunchMarks* m) {
  return a.D == 64 ? launch_prefix_t<64>(tq, tk, tv, a, qt, stream, m)
                   : launch_prefix_t<128>(tq, tk, tv, a, qt, stream, m);
}

}  // namespace fa
