"""Seeded random shapes through the grouped-head operators, against the fp64
oracles: batches, heads, lengths, masks, rotations, prefixes and pages drawn
together, so that combinations of what the hand-picked cases meet one at a
time occur too. The tolerances are those of the operators' own tests."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build
import parity_util as pu
import test_norm_rope as nr
from test_decode_shared import Step
from test_gqa_gradient_rows import reference
from test_parity_gqa import Packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def log_int(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


def heads(rng):
    Hk = int(rng.choice([1, 2, 3, 5]))
    return Hk * int(rng.choice([1, 2, 3, 4, 6, 7, 9])), Hk


@pytest.mark.parametrize("i", range(16))
def test_prompts(i):
    import torch
    rng = np.random.default_rng(51000 + i)
    H, Hk = heads(rng)
    d, causal = int(rng.choice([64, 128])), bool(rng.integers(0, 2))
    top = log_int(rng, 2, 700)
    lq = [int(rng.integers(0, top + 1)) for _ in range(int(rng.integers(1, 9)))]
    lq[int(rng.integers(len(lq)))] = top
    how = int(rng.integers(0, 3))  # keys: as many as queries, more, or drawn apart
    lk = [n + how * int(rng.integers(0, 200)) if how < 2 else int(rng.integers(0, 2 * top)) for n in lq]
    lk[0] = max(lk[0], 1)
    x = Packed(lq, lk, H, Hk, d, 51000 + i, spare=int(rng.integers(0, 3)))
    x.max_q = min(x.max_q + int(rng.integers(0, 300)), x.dev["q"].shape[0])  # a loose bound
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(causal))
    T, Tk = int(x.cu_q[-1]), int(x.cu_k[-1])
    torch.cuda.synchronize()
    ro, rl = oracle.varlen_forward(x.f["q"], x.repeated("k"), x.repeated("v"), x.cu_q, x.cu_k, x.scale, causal)
    assert pu.o_err(pu.bf16_tensor_to_f64(o)[:T], ro[:T]) <= pu.O_ATOL
    assert pu.max_abs(lse.cpu().numpy()[:, :T], rl[:, :T]) <= pu.LSE_ATOL
    val, err = reference(x, causal)
    for deterministic in (False, True):
        got = binding.attention_backward_varlen_gqa(*x.qkv(), o, lse, x.dev["do"], *x.args(causal),
                                                    deterministic=deterministic)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        for name, g, r, e, n in zip(("dQ", "dK", "dV"), got, val, err, (T, Tk, Tk)):
            g = pu.bf16_tensor_to_f64(g)[:n]
            assert np.all(np.abs(g - r[:n]) <= e[:n]), (name, i)


@pytest.mark.parametrize("i", range(12))
def test_norm_and_rotation(i):
    import torch
    rng = np.random.default_rng(52000 + i)
    H, Hk = heads(rng)
    d = int(rng.choice([64, 128]))
    rot, interleaved = 16 * int(rng.integers(0, d // 16 + 1)), bool(rng.integers(0, 2))
    c = nr.Case(log_int(rng, 1, 3000), H, Hk, d, rot, 52000 + i, fused=bool(rng.integers(0, 2)))
    y = binding.qk_norm_rope(*c.args(), nr.EPS, interleaved)
    grads = binding.qk_norm_rope_backward(*c.args(), *c.g, nr.EPS, interleaved)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    for x, w, y1, g, dx, dw in zip((c.q, c.k), c.w, y, c.g, grads[:2], grads[2:]):
        x, w, g = c.f(x), c.f(w), c.f(g)
        ref = oracle.norm_rope_forward(x, w, *c.tab, c.pos, nr.EPS, interleaved)
        assert np.all(np.abs(c.f(y1) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * c.magnitude(x, w, interleaved))
        rx, rw, _ = oracle.norm_rope_backward(x, w, *c.tab, c.pos, nr.EPS, interleaved, g)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + nr.EPS)
        du = c.spread(g, interleaved)
        dn, n = du * np.abs(w), np.abs(x) * r
        terms = r * (dn + n * np.mean(dn * n, -1, keepdims=True))
        assert np.all(np.abs(c.f(dx) - rx) <= 2.0 ** -8 * np.abs(rx) + 2.0 ** -17 * terms)
        assert np.all(np.abs(dw.cpu().numpy() - rw) <= 2.0 ** -17 * np.sum(du * n, axis=(0, 1)))


@pytest.mark.parametrize("i", range(16))
def test_decoding(i):
    import torch
    rng = np.random.default_rng(53000 + i)
    H, Hk = heads(rng)
    d, page = int(rng.choice([64, 128])), int(rng.choice([64, 128, 192, 256]))
    counts = [int(rng.integers(0, log_int(rng, 1, 40) + 1)) for _ in range(int(rng.integers(1, 5)))]
    counts[0] += 1
    before, after = (int(rng.integers(0, 3)) for _ in range(2))
    plens = [int(rng.integers(0, log_int(rng, 2, 1500))) for _ in counts]
    slens = [int(rng.integers(0, log_int(rng, 2, 400))) for _ in range(before + sum(counts) + after)]
    x = Step(counts, plens, slens, H, Hk, d, page, 53000 + i, before=before)
    # loose bounds, as far as the tables' rows reach
    x.max_p = min(x.max_p + int(rng.integers(0, 200)), x.ptab.shape[1] * page)
    x.max_s = min(x.max_s + int(rng.integers(0, 200)), x.stab.shape[1] * page)
    x.max_group = min(x.max_group + int(rng.integers(0, 3)), x.B)
    o, lse = binding.attention_decode_shared_prefix(*x.args())
    again = binding.attention_decode_shared_prefix(*x.args())
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    x.check(o, lse)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
