"""A packed batch whose middle sequence is not finite (fa_fwd_varlen,
fa_bwd_varlen and its deterministic form): its rows share tiles with those of
its neighbours, whose outputs and gradients must not change. Bit for bit, but
for dQ of the default order, which sums the same fp32 terms in another order
from run to run: two bf16 steps of the largest."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build
from test_parity_varlen import packed_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([200, 50, 129], [200, 50, 129]),
    ([5, 300, 1], [70, 300, 400]),
    ([130, 7, 300], [100, 0, 31]),      # rows that see no key before and after it
])
def test_finite_sequences_beside_one_that_is_not(lens_q, lens_k, d, causal, deterministic, bad):
    import torch
    H = 3
    cu_q, cu_k, dev, _, cu = packed_inputs(lens_q, lens_k, H, d, 6600 + d, with_do=True)
    args = (*cu, max(lens_q), max(lens_k), d ** -0.5, causal)

    def run():
        o, lse = binding.attention_forward_varlen(dev["q"], dev["k"], dev["v"], *args)
        g = binding.attention_backward_varlen(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], *args,
                                              deterministic=deterministic)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        return o, lse.T, *g

    want = run()
    for n, c in (("q", cu_q), ("do", cu_q), ("k", cu_k), ("v", cu_k)):
        dev[n][int(c[1]):int(c[2])] = bad
    got = run()
    for i, (g, w, c) in enumerate(zip(got, want, (cu_q, cu_q, cu_q, cu_k, cu_k))):
        for rows in (slice(0, int(c[1])), slice(int(c[2]), int(c[3]))):
            if i == 2 and not deterministic:
                top = float(w[rows].float().abs().max())
                assert bool(torch.isfinite(g[rows]).all())
                assert float((g[rows].float() - w[rows].float()).abs().max()) <= 2.0 ** -7 * top
            else:
                assert torch.equal(g[rows], w[rows]), i
