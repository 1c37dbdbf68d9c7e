"""Decoding steps over a 4-bit paged cache (fa_decode_paged_q4) against the
fp64 oracle on the values that the cache stands for.

Tolerances, per element of O, with W = sum of P (s code + |z|) over the keys:
  2^-8 |O|        the output's rounding (half a bf16 step at most);
  4 E W           P, off by twice the largest error E of a logit, numerator and
                  sum. A logit is d products and sums in fp32: with M the
                  largest sum of scale (s |q| code + |z| |q|) over a row's
                  elements, at most d sums of 2^-23 each: E = d 2^-23 M, plus
                  the base-2 exponential's 2^-22 and its argument's rounding
                  2^-23 max |logit|: E += 2^-22 + 2^-22 M;
  2^-11 W         p s in f16 (half a step of it);
  L 2^-30 S       terms below f16's normal numbers, 2^-14, the largest being 2^9
                  or more: 2^-25 each, 2^-34 of the largest p s <= S (the largest
                  s), times codes of up to 15;
  2^-23 (L / 32 + 64) W   fp32 sums: one for every 16 keys of a warp's share, the
                  lanes' sums of p z, the joins.
The LSE: E, and fp32 sums of up to L / 32 + 64 terms: 2^-24 (L / 32 + 64) +
2^-22 (1 + |LSE|)."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build
import parity_util as pu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


class Step:
    """A seeded step: pages scattered over the pool, garbage (NaN scales among
    it) in every slot that no sequence owns, table entries past the last page
    out of range. bound: the max_seq_len that is passed, if more than the
    longest; one of 20000 keeps every step off the clusters' way."""

    def __init__(self, lens, n_new, H, Hk, d, page, seed, q_scale=1.0, mul=1.0, bound=0):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.n, self.H, self.Hk, self.d, self.page = np.asarray(lens, np.int32), n_new, H, Hk, d, page
        self.B, self.max_len = len(lens), max(max(lens), bound, 1)
        pages = [-(-n // page) for n in lens]
        pool = sum(pages) + 2
        order = rng.permutation(pool).astype(np.int32)
        at = np.concatenate([[0], np.cumsum(pages)])
        self.table = np.full((self.B, -(-self.max_len // page)), -7, np.int32)
        codes = [rng.integers(0, 256, (pool, Hk, page, d // 2), dtype=np.uint8) for _ in range(2)]
        scales = [np.full((pool, Hk, page, d // 64, 2), NAN) for _ in range(2)]
        self.values = [[], []]
        for b, n in enumerate(lens):
            rows = order[at[b]:at[b + 1]]
            self.table[b, :len(rows)] = rows
            t = np.arange(n)
            where = (rows[t // page], slice(None), t % page)
            for i in range(2):
                x = oracle.to_bf16(rng.standard_normal((n, Hk, d)) * (mul if i else 1.0) +
                                   (0 if i else 0.5 * rng.standard_normal((Hk, d))))
                code, sz = oracle.quantise_q4(x)
                codes[i][where] = (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)
                scales[i][where] = sz
                self.values[i].append(oracle.held_q4(code, sz))
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cache = [dev(codes[0]), dev(scales[0]).to(torch.bfloat16), dev(codes[1]), dev(scales[1]).to(torch.bfloat16)]
        self.q = (dev(rng.standard_normal((self.B, n_new, H, d))) * q_scale).to(torch.bfloat16)
        self.scale = d ** -0.5

    def args(self):
        import torch
        return (self.q, *self.cache, torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda(), self.max_len,
                self.scale)

    def run(self, **kw):
        import torch
        o, lse = binding.attention_decode_paged_q4(*self.args(), **kw)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        return o, lse

    def oracle(self):
        return oracle.q4_decode_forward(pu.bf16_tensor_to_f64(self.q), *self.values, self.lens, self.scale)

    def check(self, o, lse):
        ro, rl, _ = self.oracle()
        rw = oracle.q4_decode_forward(pu.bf16_tensor_to_f64(self.q), self.values[0],
                                      [self.parts(1, b) for b in range(self.B)], self.lens, self.scale)[0]
        go, gl = pu.bf16_tensor_to_f64(o), lse.cpu().numpy().astype(np.float64)
        q, L, G = np.abs(pu.bf16_tensor_to_f64(self.q)), int(max(self.lens)), self.H // self.Hk
        M, S = 0.0, 0.0
        for b in range(self.B):
            k = self.parts(0, b)
            if len(k):
                mag = np.einsum("nhd,lhd->nhl", q[b], np.repeat(k, G, axis=1))
                M, S = max(M, self.scale * float(mag.max())), max(S, float(np.max(self.steps(1, b))))
        E = self.d * 2.0 ** -23 * M + 2.0 ** -22 + 2.0 ** -22 * M
        assert E < 0.05  # P within a fifth of itself at worst: a key left out, or one too many, still shows
        tol = 2.0 ** -8 * np.abs(ro) + (4 * E + 2.0 ** -11 + 2.0 ** -23 * (L / 32 + 64)) * rw + L * 2.0 ** -30 * S
        assert bool(np.all(np.isfinite(go))) and float(np.max(np.abs(go - ro) - tol)) <= 0
        assert np.array_equal(np.isinf(gl), np.isinf(rl)) and not np.any(np.isnan(gl))
        fin = np.isfinite(rl)
        assert np.all(np.abs(gl - rl)[fin] <= E + 2.0 ** -24 * (L / 32 + 64) + 2.0 ** -22 * (1 + np.abs(rl[fin])))
        assert np.all(go[~fin] == 0)

    def held(self, tensor, b):
        """The rows of a cache tensor that sequence b's tokens lie in, zeros where its table names no block."""
        t = np.arange(int(self.lens[b]))
        page = self.table[b, t // self.page]
        there = (page >= 0) & (page < tensor.shape[0])
        rows = tensor[np.where(there, page, 0), :, t % self.page]
        return np.where(there.reshape(-1, *[1] * (rows.ndim - 1)), rows, 0)

    def steps(self, i, b):
        return np.repeat(self.held(pu.bf16_tensor_to_f64(self.cache[2 * i + 1]), b)[..., 0], 64, -1)

    def parts(self, i, b):
        """s code + |z| of the elements of sequence b's rows."""
        sz = self.held(pu.bf16_tensor_to_f64(self.cache[2 * i + 1]), b)
        code = oracle.unpack_codes(self.held(self.cache[2 * i].cpu().numpy(), b))
        per = np.repeat(np.abs(sz), 64, -2)
        return per[..., 0] * code + per[..., 1]


CASES = [
    # lengths, n_new, H, Hk, page
    ([1], 1, 1, 1, 16),
    ([5, 0, 16, 17, 1], 1, 4, 4, 16),
    ([127, 128, 129, 63, 255], 1, 8, 2, 64),
    ([300, 1000, 2], 1, 16, 2, 48),            # pages that end inside a tile; eight heads to a key head
    ([2000, 3], 1, 9, 1, 128),                 # nine rows: two blocks of eight in one
    ([400, 77], 1, 35, 1, 256),                # three blocks of sixteen
    ([700, 33, 1, 0, 4], 5, 6, 2, 32),         # drafts, some before the first token
    ([130, 64], 7, 8, 1, 16),                  # 56 rows
    ([3000], 2, 4, 1, 64),
    ([20, 40], 33, 2, 2, 80),                  # more new queries than tokens
    ([7 * i % 513 for i in range(70)], 1, 8, 8, 64),
    ([4096, 100, 4095], 3, 12, 4, 512),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("bound", [0, 20000])
def test_against_oracle(d, case, bound):
    import torch
    lens, n, H, Hk, page = CASES[case]
    x = Step(lens, n, H, Hk, d, page, 8100 + 10 * case + d, bound=bound)
    o, lse = x.run()
    x.check(o, lse)
    again = x.run()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_one_query_without_its_axis(d):
    import torch
    x = Step([100, 3], 1, 8, 2, d, 16, 8300 + d)
    o, lse = x.run()
    x.q = x.q[:, 0].contiguous()
    o1, l1 = x.run()
    assert torch.equal(o[:, 0], o1) and torch.equal(lse[:, 0], l1)


@pytest.mark.gpu
@pytest.mark.parametrize("bound", [0, 20000])
@pytest.mark.parametrize("mul", [2.0 ** 60, 2.0 ** -60, 2.0 ** 120, 2.0 ** -115])
def test_values_of_any_range(mul, bound):
    x = Step([500, 40, 0], 2, 8, 2, 128, 64, 8310, mul=mul, bound=bound)
    x.check(*x.run())


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale", [2.0 ** 5, 2.0 ** -40, 0.0])
def test_queries_of_any_range(q_scale):
    """Logits of standard deviation 30 and more (one key takes nearly all the
    weight, and the maximum moves along the keys), next to nothing, and zero."""
    x = Step([900, 20], 1, 8, 2, 128, 64, 8320, q_scale=q_scale)
    x.q[..., ::7] *= 2.0 ** -12  # elements far below their row's largest
    x.check(*x.run())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bound", [0, 20000])
def test_nan_reaches_the_rows_that_see_it_and_no_other(d, bound):
    """A key or value group that reads as NaN: NaN in the rows that see the
    token (all of O and the LSE for a key, the group's elements for a value),
    the same bits as before in all others: other key heads, other sequences,
    queries before the token."""
    import torch
    lens, n, H, Hk, page = [200, 77, 5], 4, 6, 2, 32
    x = Step(lens, n, H, Hk, d, page, 8400 + d, bound=bound)
    o, lse = x.run()
    for which in (1, 3):
        for b, t in ((0, 50), (0, 197), (0, 199), (1, 76), (2, 1)):
            y = Step(lens, n, H, Hk, d, page, 8400 + d, bound=bound)
            y.cache[which][int(y.table[b, t // page]), 1, t % page, 0] = NAN
            o1, l1 = y.run()
            first = max(0, t - lens[b] + n)  # queries from here on see the token
            hit = torch.zeros(len(lens), n, H, dtype=torch.bool, device="cuda")
            hit[b, first:, H // 2:] = True
            assert torch.equal(o1[~hit], o[~hit]) and torch.equal(l1[~hit], lse[~hit])
            if which == 1:
                assert bool(o1[hit].isnan().all()) and bool(l1[hit].isnan().all())
            else:
                assert bool(o1[hit][:, :64].isnan().all()) and torch.equal(o1[hit][:, 64:], o[hit][:, 64:])
                assert torch.equal(l1, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("bound", [0, 20000])
def test_blocks_outside_the_pool_read_as_zeros(bound):
    x = Step([256, 130, 0, 64], 2, 8, 2, 128, 16, 8500, bound=bound)
    for b, p, bad in ((0, 1, x.cache[0].shape[0]), (1, 0, -1), (0, 9, 2 ** 31 - 1), (3, 3, -2 ** 31)):
        x.table[b, p] = bad
        for v in x.values:
            v[b][16 * p:16 * p + 16] = 0
    x.check(*x.run())


@pytest.mark.gpu
def test_lengths_past_their_bounds_are_cut():
    import torch
    x = Step([200, 90, 50], 1, 4, 2, 64, 64, 8510)
    full = Step([200, 200, 200], 1, 4, 2, 64, 64, 8511)
    a = list(full.args())
    want = binding.attention_decode_paged_q4(*a)
    a[6] = torch.tensor([10 ** 9, 201, -5], dtype=torch.int32, device="cuda")
    o, lse = binding.attention_decode_paged_q4(*a)
    torch.cuda.synchronize()
    assert torch.equal(o[:2], want[0][:2]) and torch.equal(lse[:2], want[1][:2])
    assert not o[2].any() and bool((lse[2] == float("-inf")).all())
    x.max_len = 256  # a bound above every length
    x.check(*x.run())


@pytest.mark.gpu
def test_pool_past_2_32_bytes():
    import torch
    Hk, d, page = 8, 128, 256
    x = Step([700, 1, 300], 1, 16, Hk, d, page, 8520)
    want = x.run()
    n = 34000  # 4.4e9 bytes of codes
    far = n - x.cache[0].shape[0]
    big = binding.kv_cache_q4(n, Hk, page, d)
    for t in big[1::2]:
        t.fill_(NAN)
    for t, s in zip(big, x.cache):
        t[far:] = s
    x.cache, x.table = list(big), np.where(x.table >= 0, x.table + far, x.table).astype(np.int32)
    o, lse = x.run()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("bound", [900, 20000])
def test_captured_and_on_two_streams(bound):
    """A captured step replayed on new queries, lengths and tables, while
    another step runs eagerly on a second stream with its own workspace."""
    import torch
    xs = [Step([m, 40, 0, 129], 2, 8, 2, 128, 64, 8600 + m, bound=bound) for m in (900, 350)]
    other = Step([i for i in range(40)], 1, 16, 2, 64, 64, 8650)
    want, want_other = [x.run() for x in xs], other.run()
    pool = max(x.cache[0].shape[0] for x in xs)
    bufs = list(xs[0].args())
    for i in range(1, 5):
        bufs[i] = torch.zeros((pool, *bufs[i].shape[1:]), dtype=bufs[i].dtype, device="cuda")
    o, lse = torch.empty_like(bufs[0]), torch.empty(4, 2, 8, device="cuda")
    ws = torch.empty(binding.fa_decode_paged_q4_workspace_size(4, 2, 8, 2, 128, bound), dtype=torch.uint8, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    step = lambda: binding.fa_decode_paged_q4(*bufs[:5], o, lse, *bufs[5:], ws, s1)  # noqa: E731
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
            got_other = binding.attention_decode_paged_q4(*other_args)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        for a, b in zip((o, lse, *got_other), (*w, *want_other)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_call_allocates_nothing():
    import torch
    for d in (64, 128):
        for lens, n, H in (([900, 40], 1, 8), ([300], 7, 4)):
            x = Step(lens, n, H, 2, d, 16, 8700 + d)
            x.check(*x.run())
            a, o, lse = x.args(), torch.empty_like(x.q), torch.empty(*x.q.shape[:-1], device="cuda")
            ws = torch.empty(binding.fa_decode_paged_q4_workspace_size(len(lens), n, H, 2, d, x.max_len), dtype=torch.uint8,
                             device="cuda")
            torch.cuda.synchronize()
            free = torch.cuda.mem_get_info()[0]
            for _ in range(3):
                binding.fa_decode_paged_q4(*a[:5], o, lse, *a[5:], ws)
            torch.cuda.synchronize()
            assert torch.cuda.mem_get_info()[0] == free
            x.check(o, lse)


FAKE = 0x10000
GOOD = dict(q=FAKE, kc=FAKE, lens=FAKE, o=FAKE, B=4, n=2, H=8, Hk=2, d=64, nb=10, bs=16, mb=4, ms=64, scale=0.1)


@pytest.mark.parametrize("change,expect", [
    (dict(q=None), binding.FA_ERR_INVALID),
    (dict(kc=None), binding.FA_ERR_INVALID),
    (dict(lens=None), binding.FA_ERR_INVALID),
    (dict(B=0), binding.FA_ERR_INVALID),
    (dict(n=0), binding.FA_ERR_INVALID),
    (dict(H=0), binding.FA_ERR_INVALID),
    (dict(Hk=3), binding.FA_ERR_INVALID),
    (dict(nb=0), binding.FA_ERR_INVALID),
    (dict(mb=0), binding.FA_ERR_INVALID),
    (dict(ms=0), binding.FA_ERR_INVALID),
    (dict(ms=65), binding.FA_ERR_INVALID),
    (dict(scale=0.0), binding.FA_ERR_INVALID),
    (dict(scale=float("inf")), binding.FA_ERR_INVALID),
    (dict(bs=24), binding.FA_ERR_UNSUPPORTED),
    (dict(d=256), binding.FA_ERR_UNSUPPORTED),
    (dict(nb=1 << 27), binding.FA_ERR_UNSUPPORTED),
    (dict(n=1 << 29), binding.FA_ERR_UNSUPPORTED),
    (dict(o=FAKE + 2), binding.FA_ERR_UNSUPPORTED),
    (dict(kc=FAKE + 8), binding.FA_ERR_UNSUPPORTED),
])
def test_refusals(change, expect):
    a = {**GOOD, **change}
    assert binding.load_library().fa_decode_paged_q4(
        a["q"], a["kc"], FAKE, FAKE, FAKE, a["o"], FAKE, FAKE, a["lens"], a["B"], a["n"], a["H"], a["Hk"], a["d"],
        a["nb"], a["bs"], a["mb"], a["ms"], a["scale"], FAKE, 1 << 60, None) == expect


def test_refuses_a_small_workspace():
    lib = binding.load_library()
    need = lib.fa_decode_paged_q4_workspace_size(4, 2, 8, 2, 64, 64)
    assert need > 0
    call = lambda ws, n: lib.fa_decode_paged_q4(*([FAKE] * 9), 4, 2, 8, 2, 64, 10, 16, 4, 64, 0.1, ws, n, None)  # noqa: E731
    assert call(FAKE, need - 1) == binding.FA_ERR_WORKSPACE
    assert call(None, need) == binding.FA_ERR_WORKSPACE
    assert call(FAKE + 8, need) == binding.FA_ERR_WORKSPACE
    assert lib.fa_decode_paged_q4_workspace_size(4, 2, 8, 3, 64, 64) == 0
