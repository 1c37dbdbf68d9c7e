"""Decoding for a batch that shares prefixes (fa_decode_shared_prefix) against
the fp64 oracle (prefix and own keys concatenated, one plain softmax).

Tolerances: the output's bf16 rounding (half a step) plus 2^-10 A per element,
A = sum of P |V|: P is rounded to 11 bits or better (2^-11 of each term) and a
logit is a sum of d products in fp32, off by at most d 2^-24 sum |q k| scale <
2^-12 for the seeded normal inputs, as much again relative in P. The LSE is off
by at most the logits' 2^-12 and its own rounding: 2^-11."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build, synth
import parity_util as pu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def test_oracle_without_prefix_is_paged_decoding():
    rng = np.random.default_rng(5)
    B, H, d, bs = 3, 2, 64, 64
    q, kp, vp = rng.standard_normal((B, H, d)), rng.standard_normal((7, bs, H, d)), rng.standard_normal((7, bs, H, d))
    table, lens = np.array([[4, 2], [0, 6], [1, 3]]), np.array([100, 0, 64])
    want = oracle.paged_decode_forward(q, kp, vp, table, lens, 0.125)
    none = (np.zeros((1, 1), int), np.array([0]), np.array([0, 0]))
    got = oracle.shared_prefix_decode_forward(q, kp, vp, *none, table, lens, 0.125)
    assert np.allclose(got[0], want[0]) and np.array_equal(np.isinf(got[1]), np.isinf(want[1]))
    # the first 64 own tokens of sequence 0 as its prefix: the same keys
    own = np.array([[2, 0], [0, 6], [1, 3]])
    part = oracle.shared_prefix_decode_forward(q, kp, vp, np.array([[4]]), np.array([64]), np.array([0, 1]), own,
                                               np.array([36, 0, 64]), 0.125)
    assert np.allclose(part[0], want[0])
    assert np.allclose(part[1][0], want[1][0])


class Step:
    """A seeded step: pages scattered over the pool, everything unowned NaN."""

    def __init__(self, counts, plens, slens, H, Hk, d, page, seed, before=0, q_scale=1.0):
        import torch
        self.B, self.H, self.Hk, self.d, self.page = len(slens), H, Hk, d, page
        self.plens, self.slens = np.asarray(plens, np.int32), np.asarray(slens, np.int32)
        self.cu = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
        self.max_group = max(max(counts), 1)
        self.max_p, self.max_s = max(max(plens), 1), max(max(slens), 1)
        pages = [-(-n // page) for n in (*plens, *slens)]
        pool = sum(pages) + 2
        order = np.random.default_rng(seed).permutation(pool).astype(np.int32)
        at = np.concatenate([[0], np.cumsum(pages)])
        rows = [order[at[i]:at[i + 1]] for i in range(len(pages))]
        P = len(plens)

        def table(rs, lens, width):
            t = np.full((len(rs), width), -7, np.int32)  # entries past the last page are not read
            for i, r in enumerate(rs):
                t[i, :len(r)] = r
            return t

        self.ptab = table(rows[:P], plens, -(-self.max_p // page))
        self.stab = table(rows[P:], slens, -(-self.max_s // page))
        q = synth.bf16_bits_to_f64(synth.bf16_normal_tensor(seed, synth.STREAM_Q, (self.B, H, d))) * q_scale
        self.q = torch.from_numpy(q).to(torch.bfloat16).cuda()
        bits = [synth.bf16_normal_tensor(seed, st, (pool, page, Hk, d)) for st in (synth.STREAM_K, synth.STREAM_V)]
        own = np.zeros((pool, page), bool)
        for r, n in zip(rows, (*plens, *slens)):
            for i, x in enumerate(r):
                own[x, :max(0, min(page, n - i * page))] = True
        for b in bits:
            b[~own] = 0x7FC0  # NaN
        self.f = [synth.bf16_bits_to_f64(b) for b in bits]
        self.k, self.v = (pu.to_device(b) for b in bits)
        self.scale = 1 / np.sqrt(d)

    def args(self):
        import torch
        return (self.q, self.k, self.v, *(torch.from_numpy(x).cuda() for x in
                                          (self.ptab, self.plens, self.cu, self.stab, self.slens)),
                self.max_group, self.max_p, self.max_s, self.scale)

    def oracle(self):
        return oracle.shared_prefix_decode_forward(pu.bf16_tensor_to_f64(self.q), *self.f, self.ptab, self.plens, self.cu,
                                                   self.stab, self.slens, self.scale)

    def check(self, o, lse, ref=None):
        ro, rl, ra = ref or self.oracle()
        go, gl = pu.bf16_tensor_to_f64(o), lse.cpu().numpy().astype(np.float64)
        assert np.all(np.isfinite(go))
        assert np.all(np.abs(go - ro) <= pu.bf16_half_ulp(ro) + 2.0 ** -10 * ra)
        assert pu.max_abs(gl, rl) <= 2.0 ** -11


CASES = [
    # (sequences of each prefix, prefix lengths, own lengths, H, Hk, page)
    ([4], [1000], [0, 200, 64, 1], 8, 2, 64),
    ([2, 0, 3], [65, 500, 0], [0, 63, 0, 65, 128], 6, 2, 128),   # an empty prefix, one that nobody shares
    ([1, 1], [1, 64], [1, 0], 3, 3, 64),                           # full heads, shortest lengths
    ([5], [129], [257, 0, 1, 2, 300], 16, 1, 256),                 # 80 rows: two row blocks
    ([3], [700], [64, 65, 0], 40, 1, 64),                          # 40 heads of a group on own tokens
    ([2], [300], [10, 500], 140, 2, 64),                           # 70 heads: two row blocks on own tokens
    ([9, 30], [2000, 900], [7 * i % 90 for i in range(39)], 8, 1, 64),  # up to 240 rows
    ([64], [3000], [i for i in range(64)], 8, 2, 64),              # 256 rows
    ([70], [129], [1] * 70, 12, 4, 128),                           # 210 rows, short prefix
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_oracle(d, case):
    import torch
    counts, plens, slens, H, Hk, page = CASES[case]
    x = Step(counts, plens, slens, H, Hk, d, page, 9700 + 10 * case + d)
    o, lse = binding.attention_decode_shared_prefix(*x.args())
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    x.check(o, lse)
    again = binding.attention_decode_shared_prefix(*x.args())
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_empty_sequences_and_sequences_of_no_prefix(d):
    """The first two and the last sequence belong to no prefix; sequence 0 has
    no keys at all: O = 0, LSE = -inf."""
    import torch
    x = Step([2], [150], [0, 70, 30, 0, 5], 4, 2, d, 64, 9900 + d, before=2)
    o, lse = binding.attention_decode_shared_prefix(*x.args())
    torch.cuda.synchronize()
    x.check(o, lse)
    assert bool((o[0] == 0).all()) and bool((lse[0] == float("-inf")).all())


@pytest.mark.gpu
def test_without_prefix_equals_paged_decoding():
    """Full heads, no prefix: within the tolerances of both kernels of the
    plain paged step on the same cache (which is given zeros where no sequence
    has written: it multiplies those values by zero, so they must be finite)."""
    import torch
    x = Step([0], [0], [300, 64, 1, 700], 3, 3, 128, 64, 9950)
    o, lse = binding.attention_decode_shared_prefix(*x.args())
    a = x.args()
    po, pl = binding.attention_decode_paged(a[0], a[1].nan_to_num(), a[2].nan_to_num(), a[6], a[7], x.max_s, x.scale)
    torch.cuda.synchronize()
    x.check(o, lse)
    assert (o.float() - po.float()).abs().max().item() <= 2 * 2.0 ** -8 * po.float().abs().max().item()
    assert (lse - pl).abs().max().item() <= 2.0 ** -10


@pytest.mark.gpu
@pytest.mark.parametrize("mul", [2.0 ** 40, 2.0 ** -40])
def test_values_of_any_range(mul):
    """V far outside f16's range, for few and for many rows of a prefix."""
    import torch
    for counts, slens in (([2], [40, 0]), ([40], [i % 3 for i in range(40)])):
        x = Step(counts, [500], slens, 8, 2, 128, 64, 9960)
        x.v = (x.v.float() * mul).to(torch.bfloat16)
        o, lse = binding.attention_decode_shared_prefix(*x.args())
        torch.cuda.synchronize()
        x.check(o.float() / mul, lse)


@pytest.mark.gpu
def test_sharp_softmax():
    """Logits of standard deviation 30: one key takes nearly all the weight,
    and the maximum moves along the keys. A logit's error grows with its
    magnitude, as q does: 30 times the tolerance's 2^-12 part."""
    import torch
    x = Step([40], [900], [20 + i for i in range(40)], 8, 2, 128, 64, 9970, q_scale=30.0)
    o, lse = binding.attention_decode_shared_prefix(*x.args())
    torch.cuda.synchronize()
    ro, rl, ra = x.oracle()
    assert np.all(np.abs(pu.bf16_tensor_to_f64(o) - ro) <= pu.bf16_half_ulp(ro) + 30 * 2.0 ** -10 * ra)
    assert pu.max_abs(lse.cpu().numpy(), rl) <= 30 * 2.0 ** -11


@pytest.mark.gpu
def test_blocks_outside_the_pool_read_as_zeros():
    import torch
    x = Step([3], [256], [130, 0, 64], 8, 2, 128, 64, 9980)
    want = [t.copy() for t in x.f]
    for t, i, j in ((x.ptab, 0, 1), (x.stab, 0, 0)):
        for f in want:
            f[t[i, j]] = 0
    for p, s in ((x.k.shape[0], -1), (2 ** 31 - 1, -2 ** 31)):
        y = x
        ptab, stab = x.ptab.copy(), x.stab.copy()
        x.ptab[0, 1], x.stab[0, 0] = p, s
        o, lse = binding.attention_decode_shared_prefix(*y.args())
        torch.cuda.synchronize()
        x.ptab, x.stab = ptab, stab
        ref = oracle.shared_prefix_decode_forward(pu.bf16_tensor_to_f64(x.q), *want, x.ptab, x.plens, x.cu, x.stab,
                                                  x.slens, x.scale)
        x.check(o, lse, ref)


@pytest.mark.gpu
def test_lengths_and_groups_past_their_bounds_are_cut():
    import torch
    x = Step([3, 2], [200, 100], [50, 60, 70, 80, 90], 4, 2, 64, 64, 9985)
    a = list(x.args())
    long = list(a)
    long[4], long[7] = a[4] + 10 ** 6, a[7] * 0 - 5                   # prefix lengths too long, own lengths negative
    long[5] = torch.tensor([-3, 3, 900], dtype=torch.int32, device="cuda")
    o, lse = binding.attention_decode_shared_prefix(*long)
    x.plens, x.slens = np.full(2, x.max_p, np.int32), np.zeros(5, np.int32)
    x.ptab[1] = np.where(x.ptab[1] < 0, 0, x.ptab[1])
    a = list(x.args())
    a[4] = torch.tensor([200, 200], dtype=torch.int32, device="cuda")
    want = binding.attention_decode_shared_prefix(*a[:3], a[3], a[4], a[5], a[6], a[7], *a[8:])
    torch.cuda.synchronize()
    assert torch.equal(lse[:3], want[1][:3]) and torch.equal(o[:3], want[0][:3])


@pytest.mark.gpu
def test_pool_past_2_31_elements():
    """Pages at the far end of a pool of 2.2e9 elements, NaN elsewhere."""
    import torch
    Hk, d, page = 8, 128, 512
    n = 4200
    x = Step([3], [700], [600, 1, 0], 16, Hk, d, page, 9990)
    k, v = (torch.full((n, page, Hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far = n - x.k.shape[0]
    k[far:], v[far:] = x.k, x.v
    a = list(x.args())
    a[1], a[2] = k, v
    a[3], a[6] = (torch.where(t >= 0, t + far, t) for t in (a[3], a[6]))
    o, lse = binding.attention_decode_shared_prefix(*a)
    torch.cuda.synchronize()
    x.check(o, lse)


@pytest.mark.gpu
def test_captured_and_on_two_streams():
    """A captured step replayed on new queries, lengths and tables, while
    another step runs eagerly on a second stream with its own workspace."""
    import torch
    xs = [Step([3, 5], [n, 400], [20, 0, 90, 64, 1, 2, 3, 130], 8, 2, 128, 64, 9995 + n) for n in (900, 350)]
    xs[1].max_p = 900
    wide = np.full((2, 15), -7, np.int32)
    wide[:, :xs[1].ptab.shape[1]] = xs[1].ptab
    xs[1].ptab = wide
    other = Step([40], [700], [i for i in range(40)], 16, 2, 64, 64, 9999)
    want = [binding.attention_decode_shared_prefix(*x.args()) for x in xs]
    want_other = binding.attention_decode_shared_prefix(*other.args())
    pool = max(x.k.shape[0] for x in xs)
    bufs = list(xs[0].args())
    for i in (1, 2):
        bufs[i] = torch.full((pool, *bufs[i].shape[1:]), float("nan"), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(bufs[0]), torch.empty(8, 8, device="cuda")
    ws = torch.empty(binding.fa_decode_shared_prefix_workspace_size(2, 8, 8, 2, 128, 5, 900, 130), dtype=torch.uint8,
                     device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    step = lambda: binding.fa_decode_shared_prefix(*bufs[:3], o, lse, *bufs[3:], ws, s1)  # noqa: E731
    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        step()
    other_args = other.args()
    for x, w in zip(xs, want):
        for dst, src in zip(bufs, x.args()):
            if isinstance(dst, torch.Tensor):
                dst[:src.shape[0]].copy_(src)
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graph.replay()
        with torch.cuda.stream(s2):
            got_other = binding.attention_decode_shared_prefix(*other_args)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        for a, b in zip((o, lse, *got_other), (*w, *want_other)):
            assert torch.equal(a, b)


FAKE = 0x10000
GOOD = dict(ptr=FAKE, o=FAKE, P=1, B=4, H=8, Hk=2, d=64, nb=10, bs=64, mpb=4, mb=4, mg=4, mp=200, ms=256, scale=0.1)


@pytest.mark.parametrize("change,expect", [
    (dict(ptr=None), binding.FA_ERR_INVALID),
    (dict(P=0), binding.FA_ERR_INVALID),
    (dict(B=0), binding.FA_ERR_INVALID),
    (dict(Hk=3), binding.FA_ERR_INVALID),
    (dict(nb=0), binding.FA_ERR_INVALID),
    (dict(mg=5), binding.FA_ERR_INVALID),
    (dict(mg=0), binding.FA_ERR_INVALID),
    (dict(mp=0), binding.FA_ERR_INVALID),
    (dict(mp=257), binding.FA_ERR_INVALID),
    (dict(ms=257), binding.FA_ERR_INVALID),
    (dict(scale=-1.0), binding.FA_ERR_INVALID),
    (dict(bs=32), binding.FA_ERR_UNSUPPORTED),
    (dict(d=72), binding.FA_ERR_UNSUPPORTED),
    (dict(nb=1 << 26), binding.FA_ERR_UNSUPPORTED),
    (dict(o=FAKE + 2), binding.FA_ERR_UNSUPPORTED),
])
def test_refusals(change, expect):
    lib = binding.load_library()
    a = {**GOOD, **change}
    call = lambda ws, n: lib.fa_decode_shared_prefix(  # noqa: E731
        a["ptr"], FAKE, FAKE, a["o"], *([FAKE] * 6), a["P"], a["B"], a["H"], a["Hk"], a["d"], a["nb"], a["bs"],
        a["mpb"], a["mb"], a["mg"], a["mp"], a["ms"], a["scale"], ws, n, None)
    assert call(FAKE, 1 << 40) == expect


def test_refuses_a_small_workspace():
    lib = binding.load_library()
    a = GOOD
    need = lib.fa_decode_shared_prefix_workspace_size(1, 4, 8, 2, 64, 4, 200, 256)
    assert need > 0
    call = lambda ws, n: lib.fa_decode_shared_prefix(*([FAKE] * 10), 1, 4, 8, 2, 64, 10, 64, 4, 4, 4, 200, 256, 0.1, ws, n, None)  # noqa: E731,E501
    assert call(FAKE, need - 1) == binding.FA_ERR_WORKSPACE
    assert call(None, need) == binding.FA_ERR_WORKSPACE
    assert lib.fa_decode_shared_prefix_workspace_size(1, 4, 8, 3, 64, 4, 200, 256) == 0
