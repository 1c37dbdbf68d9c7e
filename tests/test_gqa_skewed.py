"""Backward of grouped-head batches of one long and many short sequences on few
key heads: its work items are shared out over clusters of CTAs, as many as
there are key blocks in the sequences, far fewer than in the batch padded to
its longest. Every key block gets its gradients: against the fp64 oracle, and
both orders alike, bit for bit in dK and dV."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build
import parity_util as pu
from test_parity_gqa import Packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hk,d,lens_q,lens_k", [
    (4, 1, 128, [1500] + [1 + 7 * i % 60 for i in range(40)], None),
    (3, 1, 64, [20] * 12 + [1300] + [0, 5, 0], [128] * 12 + [1300] + [129, 5, 0]),  # keys without queries too
    (4, 2, 64, [129] * 19 + [900], None),                                            # the bound met: all whole + 1
])
def test_every_key_block_gets_its_gradients(H, Hk, d, lens_q, lens_k, causal):
    import torch
    x = Packed(lens_q, lens_k or lens_q, H, Hk, d, 7950)
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(causal))
    out = []
    for f in (binding.fa_bwd_varlen_gqa, binding.fa_bwd_varlen_gqa_deterministic):
        g = [torch.full_like(x.dev[n], float("nan")) for n in ("q", "k", "v")]
        f(*x.qkv(), o, lse, x.dev["do"], *g, *x.args(causal))
        out.append(g)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    assert torch.equal(out[0][1], out[1][1]) and torch.equal(out[0][2], out[1][2])
    rq, rk, rv = oracle.varlen_backward(x.f["q"], x.repeated("k"), x.repeated("v"), x.f["do"], x.cu_q, x.cu_k,
                                        x.scale, causal)
    for got in out:
        for name, g, r in (("dQ", got[0], rq), ("dK", got[1], x.grouped(rk)), ("dV", got[2], x.grouped(rv))):
            g = pu.bf16_tensor_to_f64(g)
            assert np.all(np.isfinite(g)), name
            assert pu.max_abs(g, r) <= pu.GRAD_RTOL * float(np.max(np.abs(r))), name
