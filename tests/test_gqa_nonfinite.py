"""Non-finite inputs of grouped-head prompts. A query row with a NaN logit has
NaN in O and in its LSE (an LSE of -inf means a row that sees no key), and its
gradients reach every key that it sees as NaN; other sequences and other heads
keep their bits, forward and backward (deterministic order)."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build
from test_parity_gqa import Packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def run(x, causal):
    import torch
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(causal))
    g = binding.attention_backward_varlen_gqa(*x.qkv(), o, lse, x.dev["do"], *x.args(causal), deterministic=True)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    return (o, lse, *g)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,Hk,d,causal,lens", [
    (8, 2, 128, True, [200, 131, 70]),
    (6, 2, 64, False, [200, 131, 70]),
    (4, 1, 128, True, [900, 700]),        # few key blocks: shared out over clusters
])
def test_a_bad_query_row(H, Hk, d, causal, lens, bad):
    """Element `bad` in row 40, head 1 of sequence 1 (inf: the logits of the
    row are infinite, that of key 10 is +inf)."""
    import torch
    x = Packed(lens, lens, H, Hk, d, 8900)
    x.dev["k"][lens[0] + 10, 0, 3] = 1.0
    want = run(x, causal)
    row, head, G = lens[0] + 40, 1, H // Hk
    x.dev["q"][row, head, 3] = bad
    o, lse, dq, dk, dv = run(x, causal)
    assert bool(torch.isnan(o[row, head]).all()) and bool(torch.isnan(lse[head, row]))
    assert bool(torch.isnan(dq[row, head]).all())
    seen = slice(lens[0], lens[0] + (41 if causal else lens[1]))
    assert bool(torch.isnan(dk[seen, head // G]).all()) and bool(torch.isnan(dv[seen, head // G]).all())
    # Every other row of O, LSE and dQ; every gradient of other key heads and sequences.
    wo, wl, wq, wk, wv = want
    keep = torch.ones(sum(lens), H, dtype=torch.bool, device="cuda")
    keep[row, head] = False
    assert torch.equal(o[keep], wo[keep]) and torch.equal(lse.T[keep], wl.T[keep])
    assert torch.equal(dq[keep], wq[keep])
    keep = torch.ones(sum(lens), Hk, dtype=torch.bool, device="cuda")
    keep[lens[0]:lens[0] + lens[1], 0] = False
    assert torch.equal(dk[keep], wk[keep]) and torch.equal(dv[keep], wv[keep])


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_no_key_stay_empty(d):
    """More queries than keys, bottom-right causal: the first rows see nothing; O = 0, LSE = -inf, no gradient."""
    import torch
    x = Packed([300, 50], [100, 0], 7, 1, d, 8950)
    o, lse, dq, dk, dv = run(x, True)
    none = slice(0, 200)
    assert bool((o[none] == 0).all()) and bool((lse[:, none] == float("-inf")).all()) and bool((dq[none] == 0).all())
    assert bool((o[300:] == 0).all()) and bool((lse[:, 300:] == float("-inf")).all()) and bool((dq[300:] == 0).all())
    assert all(bool(torch.isfinite(t).all()) for t in (o, dq, dk, dv))
