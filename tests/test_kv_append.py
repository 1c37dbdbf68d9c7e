"""Tokens appended to a paged cache (fa_kv_append, fa_kv_append_q4) and read
back (fa_kv_gather_q4). The rotation, the rounding and the 4-bit codes are
defined down to the last bit, so everything here is compared exactly."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build
import parity_util as pu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


# ------------------------------------------------------------------ the oracle
def test_oracle_rounds_to_bf16_as_torch_does():
    import torch
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(2000) * 10.0 ** rng.integers(-42, 38, 2000),
                        [0.0, -0.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 3.4e38, -3.4e38, np.inf, np.nan, 1e-45]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(oracle.to_bf16(x), want, equal_nan=True)


def test_oracle_codes_are_the_nearest():
    """Every element is within half a step of what its code stands for (the top
    one within a step's rounding more: 15 s may fall short of the range by
    15 * 2^-9 s)."""
    rng = np.random.default_rng(2)
    x = oracle.to_bf16(rng.standard_normal((500, 128)) * np.exp2(rng.integers(-20, 20, (500, 1))))
    codes, sz = oracle.quantise_q4(x)
    s = np.repeat(sz[..., 0], 64, -1)
    off = np.abs(oracle.held_q4(codes, sz) - x)
    assert np.all(off <= s * (0.5 + 15 * 2.0 ** -8) + 1e-300) and codes.min() == 0 and codes.max() == 15
    assert np.mean(off <= 0.5 * s * (1 + 1e-9)) > 0.97


def test_oracle_scale_through_fp32_is_the_exact_quotient():
    """bf16 of the fp32 quotient (max - min) / 15 is bf16 of the exact one."""
    rng = np.random.default_rng(3)
    hi = oracle.to_bf16(rng.standard_normal(400000) * np.exp2(rng.integers(-12, 12, 400000))).astype(np.float32)
    lo = oracle.to_bf16(rng.standard_normal(400000) * np.exp2(rng.integers(-12, 12, 400000))).astype(np.float32)
    w = np.abs(hi - lo)
    assert np.array_equal(oracle.to_bf16(w / np.float32(15)), oracle.to_bf16(w.astype(np.float64) / 15))


# ------------------------------------------------------------------------ GPU
class Append:
    """A seeded batch out of a fused projection, pages scattered over a pool."""

    def __init__(self, T, H, Hk, d, rot, page, seed, interleaved=False, pad=0, span=700, values=None):
        import torch
        rng = np.random.default_rng(seed)
        self.T, self.H, self.Hk, self.d, self.page, self.interleaved = T + pad, H, Hk, d, page, interleaved
        x = rng.standard_normal((T + pad, H + 2 * Hk, d)) if values is None else values(rng, (T + pad, H + 2 * Hk, d))
        self.qkv = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = self.qkv[:, :H], self.qkv[:, H:H + Hk], self.qkv[:, H + Hk:]
        angle = rng.uniform(-8, 8, (span, rot // 2))
        self.tab = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        self.cos, self.sin = (torch.from_numpy(t).cuda() for t in self.tab)
        self.pos = rng.integers(0, span, T + pad).astype(np.int32)
        self.blocks = -(-T // page) + 3
        self.slots = np.concatenate([rng.permutation(self.blocks * page)[:T], -1 - rng.integers(0, 9, pad)]).astype(np.int32)
        rng.shuffle(self.slots)
        self.dev = [torch.from_numpy(t).cuda() for t in (self.pos, self.slots)]

    def args(self):
        return self.q, self.k, self.v, self.cos, self.sin, *self.dev

    def rotated(self, x):
        return oracle.rotated(pu.bf16_tensor_to_f64(x), *self.tab, self.pos, self.interleaved)

    def expect(self, cache, rows):
        """cache [blocks, page, Hk, ...] with the rows put in their slots."""
        out = cache.copy().reshape(-1, *cache.shape[2:])
        on = self.slots >= 0
        out[self.slots[on]] = rows[on]
        return out.reshape(cache.shape)


def bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy()


def same(t, want):
    """A bf16 tensor against float64 values, NaN equal to NaN, zeros of either sign."""
    return np.array_equal(pu.bf16_tensor_to_f64(t), want, equal_nan=True)


CASES = [
    # T, H, Hk, d, rot, page, interleaved, pad
    (1, 1, 1, 64, 64, 16, False, 0),
    (1, 5, 1, 128, 128, 64, True, 0),
    (3, 7, 7, 128, 48, 7, False, 2),
    (17, 4, 2, 64, 16, 16, True, 0),
    (130, 12, 4, 64, 32, 48, False, 9),
    (255, 32, 8, 128, 128, 64, False, 1),
    (700, 9, 3, 128, 64, 128, True, 30),
    (40, 3, 1, 64, 0, 16, False, 3),
    (1500, 16, 5, 128, 128, 256, False, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case):
    import torch
    T, H, Hk, d, rot, page, inter, pad = CASES[case]
    x = Append(T, H, Hk, d, rot, page, 9100 + case, inter, pad)
    caches = [torch.randn(x.blocks, page, Hk, d, device="cuda").to(torch.bfloat16) for _ in range(2)]
    before = [bits(c) for c in caches]
    given = bits(x.qkv)
    q = binding.kv_append(*x.args(), *caches, inter)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    assert same(q, x.rotated(x.q)) and np.array_equal(bits(x.qkv), given)
    k = torch.from_numpy(x.rotated(x.k)).to(torch.bfloat16)
    for cache, old, rows in zip(caches, before, (bits(k), bits(x.v))):
        want = x.expect(old, rows)
        assert np.array_equal(bits(cache) & 0x7FFF, want & 0x7FFF)  # but for the sign of a zero
        assert np.array_equal(bits(cache)[want & 0x7FFF != 0], want[want & 0x7FFF != 0])


@pytest.mark.gpu
@pytest.mark.parametrize("case", [i for i in range(len(CASES)) if CASES[i][5] % 16 == 0])
def test_append_q4_and_gather(case):
    import torch
    T, H, Hk, d, rot, page, inter, pad = CASES[case]
    check_q4(Append(T, H, Hk, d, rot, page, 9200 + case, inter, pad))


def check_q4(x):
    import torch
    cache = binding.kv_cache_q4(x.blocks, x.Hk, x.page, x.d)
    for t in cache:
        t.view(torch.uint8).random_(0, 256)
    before = [t.clone() for t in cache]
    q = binding.kv_append_q4(*x.args(), *cache, x.interleaved)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    assert same(q, x.rotated(x.q))
    values = []
    for rows, codes, scales, c0, s0 in ((x.rotated(x.k), *cache[:2], *before[:2]),
                                        (pu.bf16_tensor_to_f64(x.v), *cache[2:], *before[2:])):
        want, sz = oracle.quantise_q4(rows)
        # Heads lie in front of a block's tokens.
        as_slots = lambda t: t.transpose(1, 2).contiguous()  # noqa: E731
        got = oracle.unpack_codes(as_slots(codes).cpu().numpy())
        assert np.array_equal(got, x.expect(oracle.unpack_codes(as_slots(c0).cpu().numpy()), want))
        got_sz = pu.bf16_tensor_to_f64(as_slots(scales))
        assert np.array_equal(got_sz, x.expect(pu.bf16_tensor_to_f64(as_slots(s0)), sz), equal_nan=True)
        values.append(oracle.held_q4_bf16(got, got_sz))
    # Read back as sequences of whole and broken pages, from somewhere inside.
    rng = np.random.default_rng(5)
    B = 4
    width = 3
    table = rng.integers(0, x.blocks, (B, width)).astype(np.int32)
    starts = rng.integers(0, 2 * x.page, B).astype(np.int32)
    lens = np.array([0, 1, width * x.page - starts[2], rng.integers(1, x.page)])
    starts[1] = width * x.page - 1
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    total = cu[-1] + 5  # rows of no sequence behind
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    for first in (starts, None):
        k, v = (torch.full((total, x.Hk, x.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        binding.fa_kv_gather_q4(*cache, i32(table), None if first is None else i32(first), i32(cu), k, v)
        torch.cuda.synchronize()
        for got, val in zip((k, v), values):
            want = np.full((total, x.Hk, x.d), 7.0)
            for b in range(B):
                at = (0 if first is None else first[b]) + np.arange(lens[b])
                want[cu[b]:cu[b + 1]] = val[table[b, at // x.page], at % x.page]
            assert same(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_q4_of_unusual_rows(d):
    """Constant rows, one value apart, subnormals, the largest numbers, ties
    between two codes, tiny values beside a symmetric range, NaN, infinities."""
    def values(rng, shape):
        x = rng.standard_normal(shape)
        f = x.reshape(-1, 64)
        n = len(f)
        kinds = [lambda r: np.full(64, 3.0), lambda r: np.where(r > 0, 1.0, 1.0 + 2.0 ** -7), lambda r: r * 2.0 ** -130,
                 lambda r: r * 1e-38, lambda r: r * 5e37, lambda r: np.sign(r) * 3.3e38,
                 lambda r: np.concatenate([[-7.5, 7.5], rng.integers(-15, 16, 62) / 2]),
                 lambda r: np.concatenate([[-7.5, 7.5], r[2:] * 1e-30]),
                 lambda r: np.concatenate([[0.0, 15 * 1.2109375], rng.integers(0, 31, 62) * 1.2109375 / 2]),
                 lambda r: np.where(np.arange(64) == 5, np.nan, r), lambda r: np.where(np.arange(64) == 63, np.inf, r),
                 lambda r: np.where(np.arange(64) == 0, -np.inf, r), lambda r: np.zeros(64), lambda r: -np.abs(r) * 100,
                 lambda r: np.concatenate([[-2.0 ** 20], r[1:]]), lambda r: r]
        for i in range(n):
            f[i] = kinds[i % len(kinds)](f[i])
        return x
    with np.errstate(all="ignore"):
        check_q4(Append(60, 2, 3, d, 0, 16, 9300 + d, values=values))
        check_q4(Append(60, 2, 3, d, d // 2, 32, 9310 + d, values=values))


@pytest.mark.gpu
def test_elements_past_the_rotation_are_copied_bit_for_bit():
    """Infinities, NaN and negative zeros behind the rotated part, and in rows
    that are only copied."""
    import torch
    x = Append(20, 2, 2, 128, 32, 16, 9400)
    x.qkv[:, :, 32:40] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0] * 2, device="cuda").to(torch.bfloat16)
    kc, vc = (torch.zeros(x.blocks, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = binding.kv_append(*x.args(), kc, vc)
    torch.cuda.synchronize()
    assert np.array_equal(bits(q)[..., 32:], bits(x.q)[..., 32:])
    assert np.array_equal(bits(kc.view(-1, 2, 128))[x.slots][..., 32:], bits(x.k)[..., 32:])
    assert np.array_equal(bits(vc.view(-1, 2, 128))[x.slots], bits(x.v))


@pytest.mark.gpu
def test_without_queries_and_without_tables():
    import torch
    x = Append(50, 4, 2, 128, 64, 16, 9500)
    caches = [[torch.zeros(x.blocks, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(3)]
    binding.kv_append(*x.args(), *caches[0])
    binding.fa_kv_append(None, *x.args()[1:], None, *caches[1])
    assert all(torch.equal(a, b) for a, b in zip(caches[0], caches[1]))
    binding.fa_kv_append(None, x.k, x.v, None, None, None, x.dev[1], None, *caches[2])
    torch.cuda.synchronize()
    assert np.array_equal(bits(caches[2][0].view(-1, 2, 128))[x.slots], bits(x.k))
    assert torch.equal(caches[2][1], caches[0][1])


@pytest.mark.gpu
def test_slots_and_positions_past_their_bounds():
    """Slots outside the pool are not written; positions are clamped."""
    import torch
    x = Append(30, 2, 2, 64, 64, 16, 9600)
    pool = x.blocks * 16
    bad = x.slots.copy()
    bad[:6] = [pool, pool + 1, 2 ** 31 - 1, -2 ** 31, -1, pool + 4000]
    pos = x.pos.copy()
    pos[10:14] = [-1, 700, 2 ** 31 - 1, -2 ** 31]
    x.slots, x.pos = np.where((bad < 0) | (bad >= pool), -1, bad), np.clip(pos, 0, 699)
    x.dev = [torch.from_numpy(t).cuda() for t in (pos, bad)]
    check_q4(x)
    caches = [torch.full((x.blocks, 16, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    before = [pu.bf16_tensor_to_f64(c) for c in caches]
    binding.kv_append(*x.args(), *caches)
    torch.cuda.synchronize()
    for c, b, rows in zip(caches, before, (x.rotated(x.k), pu.bf16_tensor_to_f64(x.v))):
        assert same(c, x.expect(b, rows))


@pytest.mark.gpu
def test_gather_of_what_is_not_there_reads_as_zeros():
    """Blocks outside the pool, tokens outside the table's row, starts before 0."""
    import torch
    x = Append(60, 1, 2, 64, 0, 16, 9700)
    cache = binding.kv_cache_q4(x.blocks, 2, 16, 64)
    for t in cache[1::2]:
        t.fill_(3.0)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.stack((i32(0, x.blocks, 1), i32(-1, 2, 2 ** 31 - 1)))
    k, v = binding.kv_gather_q4(*cache, table, i32(-3, 10), i32(0, 60, 100), 100)
    torch.cuda.synchronize()
    want = np.zeros(100)
    want[3:19] = 3.0    # tokens 0..15 in block 0, none in block `blocks`, 32..47 in block 1, none from 48 on
    want[35:51] = 3.0
    want[66:82] = 3.0   # tokens 10..15 in no block, 16..31 in block 2, none behind
    for t in (k, v):
        assert np.array_equal(pu.bf16_tensor_to_f64(t), np.broadcast_to(want[:, None, None], (100, 2, 64)))


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_caches_past_2_31_bytes_and_elements(q4):
    """Slots at the far end of a pool of more than 2^31 elements (and, in 4
    bits, 2^32 codes); strides that put a batch's rows 2^31 elements apart."""
    import torch
    Hk, d, page = 8, 128, 256
    blocks = 8500  # 2.2e9 elements
    x = Append(300, 8, Hk, d, 128, page, 9800)
    wide = torch.empty_strided((300, 24, d), (8 * 10 ** 6, d, 1), dtype=torch.bfloat16, device="cuda")
    wide.copy_(x.qkv)
    x.q, x.k, x.v = wide[:, :8], wide[:, 8:16], wide[:, 16:]
    far = (blocks - x.blocks) * page
    slots = torch.from_numpy(x.slots + np.int32(far)).cuda()
    if q4:
        cache = binding.kv_cache_q4(blocks, Hk, page, d)
        binding.kv_append_q4(*x.args()[:-1], slots, *cache)
        small = [t[blocks - x.blocks:].clone() for t in cache]
        want = binding.kv_cache_q4(x.blocks, Hk, page, d)
        binding.kv_append_q4(*x.args(), *want)
        table = torch.arange(blocks - x.blocks, blocks, dtype=torch.int32, device="cuda").view(1, -1)
        cu = torch.tensor([0, x.blocks * page], dtype=torch.int32, device="cuda")
        got = binding.kv_gather_q4(*cache, table, None, cu, x.blocks * page)
        ref = binding.kv_gather_q4(*want, table * 0 + torch.arange(x.blocks, dtype=torch.int32, device="cuda"), None, cu,
                                   x.blocks * page)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    else:
        cache = [torch.zeros(blocks, page, Hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        binding.kv_append(*x.args()[:-1], slots, *cache)
        small = [t[blocks - x.blocks:].clone() for t in cache]
        want = [torch.zeros(x.blocks, page, Hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        binding.kv_append(*x.args(), *want)
        assert same(want[0], x.expect(np.zeros(want[0].shape), x.rotated(x.k)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(small, want))
    assert all(not t[:blocks - x.blocks].any() for t in cache)


@pytest.mark.gpu
def test_4_bit_cache_past_2_31_words():
    """Slots whose codes lie more than 2^31 32-bit words (2^33 bytes, 2^34
    codes) into a 4-bit cache, written and read back."""
    import torch
    Hk, d, page, blocks = 8, 128, 256, 70000
    x = Append(300, 8, Hk, d, 128, page, 9810)
    assert (blocks - x.blocks) * Hk * page * d // 8 > 2 ** 31
    cache, want = (binding.kv_cache_q4(n, Hk, page, d) for n in (blocks, x.blocks))
    binding.kv_append_q4(*x.args()[:-1], x.dev[1] + (blocks - x.blocks) * page, *cache)
    binding.kv_append_q4(*x.args(), *want)
    assert all(torch.equal(t[blocks - x.blocks:], w) for t, w in zip(cache, want))
    for t in cache:
        for part in t[:blocks - x.blocks].split(10000):
            assert not part.any()
    cu = torch.tensor([0, x.blocks * page], dtype=torch.int32, device="cuda")
    table = torch.arange(x.blocks, dtype=torch.int32, device="cuda").view(1, -1)
    got = binding.kv_gather_q4(*cache, table + (blocks - x.blocks), None, cu, x.blocks * page)
    ref = binding.kv_gather_q4(*want, table, None, cu, x.blocks * page)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and all(t.any() for t in ref)


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    """Captured appends and gathers replayed on new tokens and slots, while the
    same calls run eagerly on a second stream on another cache."""
    import torch
    xs = [Append(100, 4, 2, 128, 128, 16, 9900 + i, pad=3) for i in range(3)]
    table = torch.arange(xs[0].blocks, dtype=torch.int32, device="cuda").view(1, -1)
    n = xs[0].blocks * 16
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")

    def step(args, caches, out, stream):
        binding.fa_kv_append(*args, out[0], *caches[0], stream=stream)
        binding.fa_kv_append_q4(*args, out[1], *caches[1], stream=stream)
        binding.fa_kv_gather_q4(*caches[1], table, None, cu, out[2], out[3], stream=stream)

    def make():
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        caches = [torch.zeros(xs[0].blocks, 16, 2, 128, **bf16) for _ in range(2)], binding.kv_cache_q4(xs[0].blocks, 2, 16, 128)
        return caches, [torch.empty(103, 4, 128, **bf16) for _ in range(2)] + [torch.empty(n, 2, 128, **bf16) for _ in range(2)]

    flat = lambda c, o: [*c[0], *c[1], *o]  # noqa: E731
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    bufs = [t.clone() for t in xs[0].args()]
    caches, out = make()
    torch.cuda.synchronize()
    step(bufs, caches, out, s1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        step(bufs, caches, out, s1)
    for x in xs[1:]:
        want, other = make(), make()
        step(x.args(), *want, None)
        step(xs[0].args(), *other, None)
        first = [t.clone() for t in flat(*other)]
        for t in flat(caches, out):
            t.zero_()
        for dst, src in zip(bufs, x.args()):
            dst.copy_(src)
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graph.replay()
        step(xs[0].args(), *other, s2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(flat(caches, out), flat(*want)))
        assert all(torch.equal(a, b) for a, b in zip(flat(*other), first))


# ------------------------------------------------------------------- refusals
FAKE = 0x10000
GOOD = dict(q=FAKE, k=FAKE, cos=FAKE, pos=FAKE, slots=FAKE, qo=FAKE, kc=FAKE, ks=FAKE, T=4, H=8, Hk=2, d=64, rot=64,
            mp=10, nb=10, bs=16, sq=512, sk=128, sv=128)


def append(q4, **change):
    a = {**GOOD, **change}
    sizes = [a[n] for n in ("T", "H", "Hk", "d", "rot", "mp", "nb", "bs", "sq", "sk", "sv")]
    lib = binding.load_library()
    head = (a["q"], a["k"], FAKE, a["cos"], FAKE, a["pos"], a["slots"], a["qo"], a["kc"])
    if q4:
        return lib.fa_kv_append_q4(*head, a["ks"], FAKE, FAKE, *sizes, 0, None)
    return lib.fa_kv_append(*head, FAKE, *sizes, 0, None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("change,expect", [
    (dict(k=None), binding.FA_ERR_INVALID),
    (dict(slots=None), binding.FA_ERR_INVALID),
    (dict(kc=None), binding.FA_ERR_INVALID),
    (dict(q=None), binding.FA_ERR_INVALID),              # q_out without q
    (dict(qo=None), binding.FA_ERR_INVALID),
    (dict(cos=None), binding.FA_ERR_INVALID),
    (dict(pos=None), binding.FA_ERR_INVALID),
    (dict(T=0), binding.FA_ERR_INVALID),
    (dict(H=0), binding.FA_ERR_INVALID),
    (dict(Hk=0), binding.FA_ERR_INVALID),
    (dict(rot=-16), binding.FA_ERR_INVALID),
    (dict(rot=80), binding.FA_ERR_INVALID),
    (dict(mp=0), binding.FA_ERR_INVALID),
    (dict(nb=0), binding.FA_ERR_INVALID),
    (dict(bs=0), binding.FA_ERR_INVALID),
    (dict(sq=504), binding.FA_ERR_INVALID),
    (dict(sk=120), binding.FA_ERR_INVALID),
    (dict(sv=120), binding.FA_ERR_INVALID),
    (dict(rot=8), binding.FA_ERR_UNSUPPORTED),
    (dict(d=96, sq=8 * 96, sk=192, sv=192), binding.FA_ERR_UNSUPPORTED),
    (dict(sq=516), binding.FA_ERR_UNSUPPORTED),
    (dict(sk=132), binding.FA_ERR_UNSUPPORTED),
    (dict(sv=1 << 40), binding.FA_ERR_UNSUPPORTED),
    (dict(nb=1 << 27), binding.FA_ERR_UNSUPPORTED),
    (dict(q=FAKE + 2), binding.FA_ERR_UNSUPPORTED),
    (dict(k=FAKE + 8), binding.FA_ERR_UNSUPPORTED),
    (dict(cos=FAKE + 4), binding.FA_ERR_UNSUPPORTED),
    (dict(kc=FAKE + 4), binding.FA_ERR_UNSUPPORTED),
])
def test_append_refusals(q4, change, expect):
    assert append(q4, **change) == expect


def test_q4_refusals():
    assert append(True, ks=None) == binding.FA_ERR_INVALID
    assert append(True, bs=24) == binding.FA_ERR_UNSUPPORTED
    assert append(True, ks=FAKE + 8) == binding.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,expect", [
    (dict(kc=None), binding.FA_ERR_INVALID),
    (dict(table=None), binding.FA_ERR_INVALID),
    (dict(cu=None), binding.FA_ERR_INVALID),
    (dict(v=None), binding.FA_ERR_INVALID),
    (dict(batch=0), binding.FA_ERR_INVALID),
    (dict(total=0), binding.FA_ERR_INVALID),
    (dict(Hk=0), binding.FA_ERR_INVALID),
    (dict(nb=0), binding.FA_ERR_INVALID),
    (dict(mb=0), binding.FA_ERR_INVALID),
    (dict(bs=40), binding.FA_ERR_UNSUPPORTED),
    (dict(d=192), binding.FA_ERR_UNSUPPORTED),
    (dict(nb=1 << 27), binding.FA_ERR_UNSUPPORTED),
    (dict(kc=FAKE + 8), binding.FA_ERR_UNSUPPORTED),
    (dict(v=FAKE + 2), binding.FA_ERR_UNSUPPORTED),
])
def test_gather_refusals(change, expect):
    a = {**dict(kc=FAKE, table=FAKE, cu=FAKE, v=FAKE, batch=2, Hk=2, d=64, total=10, nb=10, bs=16, mb=4), **change}
    assert binding.load_library().fa_kv_gather_q4(
        a["kc"], FAKE, FAKE, FAKE, a["table"], None, a["cu"], FAKE, a["v"], a["batch"], a["Hk"], a["d"], a["total"],
        a["nb"], a["bs"], a["mb"], None) == expect
