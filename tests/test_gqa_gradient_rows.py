"""Gradients of grouped-head prompts element by element: each against a bound
made of the magnitudes of its own terms, so that the small gradients of late
keys and of early queries count like the large ones (a bound relative to the
batch's largest gradient is blind to them).

The bound, for one head (u = 2^-24; all sums fp32, so n terms add n u of
their magnitudes; bf16 rounds by 2^-8 of the value, f16 by 2^-11):
  logits     e_s = scale d u |Q||K|^T, and P = exp(s - LSE) has the relative
             error r = e_s + its largest in the row (through LSE) + 2^-18 (the
             exponential, the scaled logit's and LSE's own roundings)
  O          e_O = 2^-8 |O| + (r + 2^-11) P|V| (P in f16, O stored in bf16)
  delta      e_D = |dO| e_O + d u |dO||O|
  dP         e_dP = d u |dO||V|^T
  dV         sum_i (r + 2^-8) P |dO| (P in bf16) + 2^-8 |dV| + n u P|dO|
  dS         e_dS = P (e_dP + e_D) + (r + 2^-11 + 2^-8) |dS| + 2^-35 |dP - D|
             (P in f16 scaled by 2^10: below 2^-24 an absolute 2^-35; dS in bf16)
  dQ, dK     scale (e_dS + n u |dS|) |K| or |Q| + 2^-8 of the value,
with n the number of terms (of dK and dV those of all heads of the group). A factor 1 + 2^-6 covers products of errors."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build
import parity_util as pu
from test_parity_gqa import CASES, Packed

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def head_bounds(q, k, v, do, scale, causal, G):
    """dQ, dK, dV of one head (of G that share k and v) of one sequence and
    their bounds before the last rounding (all fp64)."""
    (lq, d), lk = q.shape, k.shape[0]
    aq, ak, av, ado = (np.abs(t) for t in (q, k, v, do))
    s = scale * (q @ k.T)
    seen = np.ones((lq, lk), bool)
    if causal:
        seen = np.arange(lk) <= np.arange(lq)[:, None] + lk - lq
    s[~seen] = -np.inf
    m = np.max(s, axis=1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    z = p.sum(1, keepdims=True)
    p = p / np.where(z > 0, z, 1.0)
    o = p @ v
    dp = do @ v.T
    delta = np.sum(do * o, axis=1, keepdims=True)
    ds = p * (dp - delta)
    dq, dk, dv = scale * (ds @ k), scale * (ds.T @ q), p.T @ do

    e_s = np.where(seen, scale * d * U * (aq @ ak.T), 0.0)
    r = e_s + np.max(e_s, axis=1, keepdims=True, initial=0.0) + 2.0 ** -18
    e_o = 2.0 ** -8 * np.abs(o) + (p * (r + 2.0 ** -11)) @ av
    e_d = np.sum(ado * (e_o + d * U * np.abs(o)), axis=1, keepdims=True)
    e_dp = d * U * (ado @ av.T)
    ads = np.abs(ds)
    e_ds = p * (e_dp + e_d) + (r + 2.0 ** -11 + 2.0 ** -8) * ads + np.where(seen, 2.0 ** -35 * np.abs(dp - delta), 0.0)
    slack = 1 + 2.0 ** -6
    b_q = slack * scale * (e_ds + lk * U * ads) @ ak
    b_k = slack * scale * (e_ds + G * lq * U * ads).T @ aq
    b_v = slack * (p * (r + 2.0 ** -8 + G * lq * U)).T @ ado
    return (dq, dk, dv), (b_q, b_k, b_v)


def reference(x, causal):
    """Gradients and bounds of a packed batch, dK and dV summed over each group."""
    H, G = x.H, x.H // x.Hk
    val = [np.zeros_like(x.f[n]) for n in ("q", "k", "v")]
    err = [np.zeros_like(t) for t in val]
    for b in range(len(x.cu_q) - 1):
        a, c = slice(x.cu_q[b], x.cu_q[b + 1]), slice(x.cu_k[b], x.cu_k[b + 1])
        if x.cu_q[b] == x.cu_q[b + 1] or x.cu_k[b] == x.cu_k[b + 1]:
            continue
        for h in range(H):
            j = h // G
            g, e = head_bounds(x.f["q"][a, h], x.f["k"][c, j], x.f["v"][c, j], x.f["do"][a, h], x.scale, causal, G)
            for t, u in ((val, g), (err, e)):
                t[0][a, h] = u[0]
                t[1][c, j] += u[1]
                t[2][c, j] += u[2]
    return val, [e + 2.0 ** -8 * (np.abs(t) + e) for t, e in zip(val, err)]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_every_gradient_within_its_own_bound(d, causal, case):
    import torch
    H, Hk, lq, lk = CASES[case]
    x = Packed(lq, lk, H, Hk, d, 7300 + 19 * case + d)
    val, err = reference(x, causal)
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(causal))
    for deterministic in (False, True):
        got = binding.attention_backward_varlen_gqa(*x.qkv(), o, lse, x.dev["do"], *x.args(causal),
                                                    deterministic=deterministic)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        for name, g, r, e in zip(("dQ", "dK", "dV"), got, val, err):
            g = pu.bf16_tensor_to_f64(g)
            assert np.all(np.isfinite(g)), name
            worst = float(np.max(np.abs(g - r) / np.maximum(e, 1e-300)))
            print(name, "worst share of the bound", round(worst, 3))
            assert worst <= 1.0, (name, worst)


@pytest.mark.parametrize("d", [64, 128])
def test_the_bound_notices_zeros(d):
    """The bounds of 700 + 650 tokens on one key head: a key block of zeros
    would exceed them in every row of it, the last one included."""
    rng = np.random.default_rng(6)
    lq, G = 650, 4
    k, v = rng.standard_normal((2, lq, d))
    val, err = [np.zeros((lq, d)) for _ in range(2)], [np.zeros((lq, d)) for _ in range(2)]
    for _ in range(G):
        q, do = rng.standard_normal((2, lq, d))
        g, e = head_bounds(q, k, v, do, d ** -0.5, True, G)
        for i in (0, 1):
            val[i] += g[1 + i]
            err[i] += e[1 + i]
    for t, e in zip(val, err):
        over = np.abs(t) > e + 2.0 ** -8 * np.abs(t)
        assert np.all(np.mean(over, axis=1) > 0.5)
