"""Per-head norm of queries and keys with the rotation, forward and backward,
against the fp64 oracle (oracle/norm_rope.py), which is itself pinned here by
closed forms and finite differences.

Tolerances. The kernels compute in fp32 and round once to bf16 (half a step:
2^-8 of the value). In fp32 an output y = r (x w c + x' w' s') takes fewer than
16 roundings of 2^-24 each beside the sum of d squares (at most d / 2 of its
roundings act on one value through r, whose relative error is half the sum's:
2^-24 * d / 4 <= 2^-19), so its error is below 2^-18 of the sum of its two
terms' magnitudes. dx adds the second row sum: 2^-17 of its terms' magnitudes.
dw sums fewer than 100 roundings deep per column: 2^-17 of the sum of
magnitudes."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build, synth
import parity_util as pu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def tables(max_pos, rot):
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(max_pos)[:, None] * freq
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# ------------------------------------------------------------ the oracle's own pins
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_keeps_norms_and_relative_positions(interleaved):
    rng = np.random.default_rng(1)
    d, rot, T = 64, 32, 9
    cos, sin = (t.astype(np.float64) for t in tables(64, rot))
    x = rng.standard_normal((T, 1, d))
    pos = np.arange(T) * 3
    y = oracle.norm_rope_forward(x, np.ones(d), cos, sin, pos, 0.0, interleaved)
    # unit weight: rows have root mean square 1 before and after the rotation
    # (the tables are fp32: cos^2 + sin^2 = 1 to 1e-7)
    assert np.allclose(np.mean(y * y, axis=-1), 1.0, atol=1e-6)
    # same vector at positions p and p + 3: products depend on the distance only
    same = np.repeat(x[:1], T, axis=0)
    z = oracle.norm_rope_forward(same, np.ones(d), cos, sin, pos, 0.0, interleaved)[:, 0]
    dots = np.sum(z[1:] * z[:-1], axis=-1)
    assert np.allclose(dots, dots[0], atol=1e-5)
    # position 0 turns nothing, and elements past rot are never turned
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True))
    assert np.allclose(y[0], n[0]) and np.allclose(y[..., rot:], n[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_backward_matches_differences(interleaved):
    rng = np.random.default_rng(2)
    T, H, d, rot = 3, 2, 64, 48
    cos, sin = tables(40, rot)
    x, dy = rng.standard_normal((2, T, H, d))
    w = 1 + 0.3 * rng.standard_normal(d)
    pos = np.array([0, 7, 39])
    loss = lambda x, w: float(np.sum(oracle.norm_rope_forward(x, w, cos, sin, pos, EPS, interleaved) * dy))  # noqa: E731
    dx, dw, _ = oracle.norm_rope_backward(x, w, cos, sin, pos, EPS, interleaved, dy)
    for _ in range(4):
        u, v = rng.standard_normal(x.shape), rng.standard_normal(d)
        h = 1e-5
        diff = (loss(x + h * u, w + h * v) - loss(x - h * u, w - h * v)) / (2 * h)
        assert abs(diff - np.sum(dx * u) - np.sum(dw * v)) < 1e-6 * (1 + abs(diff))


# ------------------------------------------------------------ GPU
class Case:
    """Seeded inputs; fused: q and k are parts of one [T, (H + 2 Hk) d] tensor."""

    def __init__(self, T, H, Hk, d, rot, seed, fused=True, scale=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.T, self.H, self.Hk, self.d, self.rot = T, H, Hk, d, rot
        bits = synth.bf16_normal_tensor(seed, synth.STREAM_Q, (T, (H + 2 * Hk) * d))
        qkv = pu.to_device(bits) * scale
        q, k = qkv[:, :H * d].view(T, H, d), qkv[:, H * d:(H + Hk) * d].view(T, Hk, d)
        self.q, self.k = (q, k) if fused else (q.contiguous(), k.contiguous())
        self.w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(torch.bfloat16).cuda()
                  for _ in range(2)]
        self.max_pos = 700
        self.tab = tables(self.max_pos, rot)
        self.cos, self.sin = (torch.from_numpy(t).cuda() for t in self.tab)
        self.pos = rng.integers(0, self.max_pos, T).astype(np.int32)
        self.pos[0] = self.max_pos - 1
        self.positions = torch.from_numpy(self.pos).cuda()
        self.g = [pu.to_device(synth.bf16_normal_tensor(seed, st, (T, h, d)))
                  for st, h in ((synth.STREAM_K, H), (synth.STREAM_V, Hk))]

    def args(self):
        return self.q, self.k, *self.w, self.cos, self.sin, self.positions

    def f(self, t):
        return pu.bf16_tensor_to_f64(t)

    def spread(self, u, interleaved):
        """|u_e c_e| + |u_e' s_e|: the magnitudes of the two terms of each rotated element."""
        c, n = (np.abs(t[self.pos].astype(np.float64))[:, None] for t in self.tab)
        i, j = oracle.norm_rope._pairs(self.rot, interleaved)
        y = np.abs(u)
        y[..., i], y[..., j] = y[..., i] * c + y[..., j] * n, y[..., j] * c + y[..., i] * n
        return y

    def magnitude(self, x, w, interleaved):
        return self.spread(x * w / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS), interleaved)


SHAPES = [
    # (T, H, Hk, d, rot)
    (1, 1, 1, 64, 64),
    (1, 32, 8, 128, 128),
    (13, 7, 1, 128, 64),
    (5, 12, 4, 64, 16),
    (3, 5, 3, 64, 48),
    (333, 9, 2, 128, 96),
    (2500, 10, 3, 64, 32),   # units of eight rows, slices of 8 and 2
    (3001, 16, 4, 128, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_forward(shape, interleaved):
    import torch
    c = Case(*SHAPES[shape], 9100 + shape)
    got = binding.qk_norm_rope(*c.args(), EPS, interleaved)
    torch.cuda.synchronize()
    for x, w, y in zip((c.q, c.k), c.w, got):
        assert y.is_contiguous() and y.shape == x.shape
        x, w = c.f(x), c.f(w)
        ref = oracle.norm_rope_forward(x, w, *c.tab, c.pos, EPS, interleaved)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * c.magnitude(x, w, interleaved)
        assert np.all(np.abs(c.f(y) - ref) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_backward(shape, interleaved):
    import torch
    c = Case(*SHAPES[shape], 9200 + shape)
    got = binding.qk_norm_rope_backward(*c.args(), *c.g, EPS, interleaved)
    again = binding.qk_norm_rope_backward(*c.args(), *c.g, EPS, interleaved)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # a fixed order of every sum
    for x, w, g, dx, dw in zip((c.q, c.k), c.w, c.g, got[:2], got[2:]):
        x, w, g = c.f(x), c.f(w), c.f(g)
        rx, rw, mag = oracle.norm_rope_backward(x, w, *c.tab, c.pos, EPS, interleaved, g)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
        du = c.spread(g, interleaved)
        dn, n = du * np.abs(w), np.abs(x) * r
        terms = r * (dn + n * np.mean(dn * n, -1, keepdims=True))
        assert np.all(np.abs(c.f(dx) - rx) <= 2.0 ** -8 * np.abs(rx) + 2.0 ** -17 * terms)
        # each term of dw is du n with du = g c + g' s', whose magnitudes bound its roundings
        bound = np.sum(du * n, axis=(0, 1))
        assert np.all(np.abs(dw.cpu().numpy() - rw) <= 2.0 ** -17 * bound)


@pytest.mark.gpu
def test_strides_and_untouched_surroundings():
    """Contiguous and fused inputs give the same bits; gradients written into
    a fused buffer leave its value part as it was."""
    import torch
    T, H, Hk, d = 57, 6, 2, 128
    a, b = Case(T, H, Hk, d, 128, 9300), Case(T, H, Hk, d, 128, 9300, fused=False)
    for x, y in zip(binding.qk_norm_rope(*a.args()), binding.qk_norm_rope(*b.args())):
        assert torch.equal(x, y)
    want = binding.qk_norm_rope_backward(*b.args(), *b.g)
    buf = torch.full((T, (H + 2 * Hk) * d), 7.0, dtype=torch.bfloat16, device="cuda")
    dq, dk = buf[:, :H * d].view(T, H, d), buf[:, H * d:(H + Hk) * d].view(T, Hk, d)
    dw = [torch.empty(d, device="cuda") for _ in range(2)]
    binding.fa_qk_norm_rope_bwd(*a.args(), *a.g, dq, dk, *dw)
    torch.cuda.synchronize()
    for x, y in zip((dq, dk, *dw), want):
        assert torch.equal(x, y)
    assert bool((buf[:, (H + Hk) * d:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 50])
def test_rows_of_extreme_scale(scale):
    """Squares stay in fp32's range down to 2^-60 (the sum is then far below
    eps: a plain scaling) and up to 2^50."""
    import torch
    c = Case(9, 3, 1, 64, 64, 9400, scale=scale)
    got = binding.qk_norm_rope(*c.args(), EPS)
    torch.cuda.synchronize()
    for x, w, y in zip((c.q, c.k), c.w, got):
        x, w = c.f(x), c.f(w)
        ref = oracle.norm_rope_forward(x, w, *c.tab, c.pos, EPS, False)
        assert np.all(np.abs(c.f(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * c.magnitude(x, w, False))


@pytest.mark.gpu
def test_zero_rows_and_positions_outside_the_table():
    """A zero row gives zeros, and finite gradients; positions outside the
    table are read as its nearest row."""
    import torch
    c = Case(6, 2, 1, 128, 128, 9500)
    c.q[2] = 0
    yq, _ = binding.qk_norm_rope(*c.args())
    dq, _, _, _ = binding.qk_norm_rope_backward(*c.args(), *c.g)
    torch.cuda.synchronize()
    assert bool((yq[2] == 0).all()) and bool(torch.isfinite(dq).all())
    outside, nearest = c.positions.clone(), c.positions.clone()
    outside[0], outside[1] = c.max_pos + 5, -3
    nearest[0], nearest[1] = c.max_pos - 1, 0
    a = binding.qk_norm_rope(*c.args()[:-1], outside)
    b = binding.qk_norm_rope(*c.args()[:-1], nearest)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_captured_on_its_own_stream():
    import torch
    cs = [Case(40, 8, 2, 64, 64, 9600 + i) for i in range(2)]
    want = [(*binding.qk_norm_rope(*c.args()), *binding.qk_norm_rope_backward(*c.args(), *c.g)) for c in cs]
    base = Case(40, 8, 2, 64, 64, 9600)
    out = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in want[0]]
    ws = torch.empty(binding.fa_qk_norm_rope_bwd_workspace_size(40, 8, 2, 64), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()

    def step():
        binding.fa_qk_norm_rope(*base.args(), out[0], out[1], stream=s)
        binding.fa_qk_norm_rope_bwd(*base.args(), *base.g, *out[2:], workspace=ws, stream=s)

    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for c, w in zip(cs, want):
        for dst, src in zip((*base.args(), *base.g), (*c.args(), *c.g)):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))


@pytest.mark.gpu
def test_tensors_past_2_31_elements():
    """2.2e9 elements of q: rows at both boundaries and at the end equal the
    same tokens in a call of their own (a row depends on its token alone)."""
    import torch
    T, H, Hk, d = 540_000, 32, 1, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    src = torch.randn(1009, (H + Hk) * d, device="cuda", generator=g).to(torch.bfloat16)
    qkv = src[torch.arange(T, device="cuda") % 1009]
    q, k = qkv[:, :H * d].view(T, H, d), qkv[:, H * d:].view(T, Hk, d)
    c = Case(3, 1, 1, d, 128, 9700)
    pos = (torch.arange(T, device="cuda") % 700).to(torch.int32)
    args = (*c.w, c.cos, c.sin)
    yq, yk = binding.qk_norm_rope(q, k, *args, pos)
    dq, dk, _, _ = binding.qk_norm_rope_backward(q, k, *args, pos, yq, yk)
    for t0 in (0, 2 ** 30 // (H * d) - 50, 2 ** 31 // (H * d) - 50, 2 ** 31 // ((H + Hk) * d) - 50, T - 100):
        rows = slice(t0, t0 + 100)
        y = binding.qk_norm_rope(q[rows], k[rows], *args, pos[rows])
        x = binding.qk_norm_rope_backward(q[rows], k[rows], *args, pos[rows], *y)
        torch.cuda.synchronize()
        for a, b in zip((yq, yk, dq, dk), (*y, *x[:2])):
            assert torch.equal(a[rows], b)


# ------------------------------------------------------------ refusals (host only)
FAKE = 0x10000
GOOD = dict(ptr=FAKE, out=FAKE, T=4, H=8, Hk=2, d=64, rot=64, max_pos=10, qs=512, ks=128, eps=1e-6)


@pytest.mark.parametrize("change,expect", [
    (dict(ptr=None), binding.FA_ERR_INVALID),
    (dict(out=None), binding.FA_ERR_INVALID),
    (dict(T=0), binding.FA_ERR_INVALID),
    (dict(Hk=0), binding.FA_ERR_INVALID),
    (dict(max_pos=0), binding.FA_ERR_INVALID),
    (dict(rot=80), binding.FA_ERR_INVALID),
    (dict(rot=-16), binding.FA_ERR_INVALID),
    (dict(qs=511), binding.FA_ERR_INVALID),
    (dict(eps=-1.0), binding.FA_ERR_INVALID),
    (dict(eps=float("nan")), binding.FA_ERR_INVALID),
    (dict(d=96), binding.FA_ERR_UNSUPPORTED),
    (dict(rot=24), binding.FA_ERR_UNSUPPORTED),
    (dict(ks=132), binding.FA_ERR_UNSUPPORTED),
    (dict(qs=1 << 40), binding.FA_ERR_UNSUPPORTED),
    (dict(ptr=FAKE + 8), binding.FA_ERR_UNSUPPORTED),
    (dict(out=FAKE + 8), binding.FA_ERR_UNSUPPORTED),
])
def test_refusals(change, expect):
    lib = binding.load_library()
    a = {**GOOD, **change}
    sizes = (a["T"], a["H"], a["Hk"], a["d"], a["rot"], a["max_pos"], a["qs"], a["ks"])
    assert lib.fa_qk_norm_rope(a["ptr"], *([FAKE] * 6), a["out"], FAKE, *sizes, a["eps"], 0, None) == expect
    assert lib.fa_qk_norm_rope_bwd(a["ptr"], *([FAKE] * 8), a["out"], FAKE, FAKE, FAKE, *sizes, 512, 128, a["eps"], 0,
                                   FAKE, 1 << 40, None) == expect


def test_backward_refuses_strides_and_workspace():
    lib = binding.load_library()
    sizes = (4, 8, 2, 64, 64, 10, 512, 128)
    need = lib.fa_qk_norm_rope_bwd_workspace_size(4, 8, 2, 64)
    call = lambda dqs, ws, n: lib.fa_qk_norm_rope_bwd(*([FAKE] * 13), *sizes, dqs, 128, 1e-6, 0, ws, n, None)  # noqa: E731
    assert call(504, FAKE, need) == binding.FA_ERR_INVALID
    assert call(516, FAKE, need) == binding.FA_ERR_UNSUPPORTED
    assert call(512, FAKE, need - 1) == binding.FA_ERR_WORKSPACE
    assert call(512, None, need) == binding.FA_ERR_WORKSPACE
    assert lib.fa_qk_norm_rope_bwd_workspace_size(0, 8, 2, 64) == 0
