"""Padding of a fixed-layout batch that holds NaN or infinity: the K and V rows
past each kv_lens (fa_fwd, fa_bwd and its deterministic and allocation-free
forms). Masked keys reach no output: everything equals, bit for bit, the same
call with zeros there (dQ of the default order, whose sums run in another order
from run to run: two bf16 steps of the largest), and their own gradients are
zero."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("how", ["default", "deterministic", "noalloc"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,lens", [(300, [300, 299, 129, 128, 127, 1, 0]), (1000, [700, 1000, 513, 5])])
def test_padding_reaches_nothing(N, lens, d, causal, how, bad):
    import torch
    B, H = len(lens), 2
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    q, k, v, do = (torch.randn(B, H, N, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(4))
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pad = (torch.arange(N, device="cuda") >= kv[:, None])[:, None, :, None].expand(B, H, N, d)

    def run(fill):
        kk, vv = (t.masked_fill(pad, fill) for t in (k, v))
        o, lse = binding.attention_forward(q, kk, vv, d ** -0.5, causal, kv)
        grads = [torch.full_like(q, 7.0) for _ in range(3)]
        fn = {"default": binding.fa_bwd, "deterministic": binding.fa_bwd_deterministic,
              "noalloc": binding.fa_bwd_noalloc}[how]
        fn(q, kk, vv, o, lse, do, *grads, d ** -0.5, causal, kv)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        return o, lse, *grads

    want, got = run(0.0), run(bad)
    for i, (a, b) in enumerate(zip(got, want)):
        if i == 2 and how != "deterministic":
            assert bool(torch.isfinite(a).all())
            assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
        else:
            assert torch.equal(a, b), i
    for t in got[3:]:
        assert bool((t[pad] == 0).all())
