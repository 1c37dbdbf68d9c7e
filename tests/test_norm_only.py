"""The per-head norm without a rotation (rot = 0, empty tables), both
directions, against the fp64 oracle, with the tolerances of the norm with one
(test_norm_rope.py), and what it still refuses."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build
import test_norm_rope as nr


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,d", [(1, 1, 1, 64), (13, 7, 1, 128), (2500, 10, 3, 64)])
def test_norm_without_rotation(T, H, Hk, d, interleaved):
    import torch
    c = nr.Case(T, H, Hk, d, 0, 9450 + T)
    assert c.cos.shape == (c.max_pos, 0)
    y = binding.qk_norm_rope(*c.args(), nr.EPS, interleaved)
    grads = binding.qk_norm_rope_backward(*c.args(), *c.g, nr.EPS, interleaved)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    for x, w, y1, g, dx, dw in zip((c.q, c.k), c.w, y, c.g, grads[:2], grads[2:]):
        x, w, g = c.f(x), c.f(w), c.f(g)
        ref = oracle.norm_rope_forward(x, w, *c.tab, c.pos, nr.EPS, interleaved)
        assert np.all(np.abs(c.f(y1) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.abs(ref))
        rx, rw, mag = oracle.norm_rope_backward(x, w, *c.tab, c.pos, nr.EPS, interleaved, g)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + nr.EPS)
        dn, n = np.abs(g * w), np.abs(x) * r
        terms = r * (dn + n * np.mean(dn * n, -1, keepdims=True))
        assert np.all(np.abs(c.f(dx) - rx) <= 2.0 ** -8 * np.abs(rx) + 2.0 ** -17 * terms)
        assert np.all(np.abs(dw.cpu().numpy() - rw) <= 2.0 ** -17 * mag)


FAKE = nr.FAKE


@pytest.mark.parametrize("tables,rot,expect", [
    ((None, None), 16, binding.FA_ERR_INVALID),
    ((None, FAKE), 64, binding.FA_ERR_INVALID),
    ((FAKE, FAKE + 8), 64, binding.FA_ERR_UNSUPPORTED),
    # accepted as far as the tables go: the next check is the outputs' alignment
    ((None, None), 0, binding.FA_ERR_UNSUPPORTED),
    ((FAKE + 4, None), 0, binding.FA_ERR_UNSUPPORTED),
])
def test_tables_are_required_for_a_rotation_only(tables, rot, expect):
    lib = binding.load_library()
    sizes = (4, 8, 2, 64, rot, 10, 512, 128)
    assert lib.fa_qk_norm_rope(FAKE, FAKE, FAKE, FAKE, *tables, FAKE, FAKE + 8, FAKE, *sizes, 1e-6, 0, None) == expect
    assert lib.fa_qk_norm_rope_bwd(FAKE, FAKE, FAKE, FAKE, *tables, FAKE, FAKE, FAKE, FAKE + 8, FAKE, FAKE, FAKE,
                                   *sizes, 512, 128, 1e-6, 0, FAKE, 1 << 40, None) == expect
