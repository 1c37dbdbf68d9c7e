"""Decoding steps over a 4-bit paged cache whose CTAs go through several tiles
each, on caches made on the GPU, against the definition in 64 bits (torch).

Tolerances, per element of O, all of them of the query and head in question,
with P the softmax and W = sum of P (s code + |z|) over the keys:
  2^-8 |O|        the output's rounding (half a bf16 step at most);
  4 E W           P, off by twice the largest error E of a logit, numerator and
                  sum: d products and sums in fp32 of at most M = scale times the
                  sum of (s code + |z|) |q| each, 2^-23 of it, the base-2
                  exponential's 2^-22 and its argument's rounding 2^-22 M;
  2^-11 W         p s in f16 (half a step of it);
  L 2^-30 S       terms below f16's normal numbers, 2^-14, where the largest p s so
                  far lies at 2^9 or more: 2^-25 each, 2^-34 of S, the largest P s of
                  the row and group, times codes of up to 15;
  2^-23 (L / 32 + 64) W   fp32 sums: one for every 16 keys of a warp's share, the
                  lanes' sums of p z, the joins.
The LSE: E, and fp32 sums of up to L / 32 + 64 terms: 2^-24 (L / 32 + 64) +
2^-22 (1 + |LSE|)."""
import math

import pytest

from exact_io_aware_29_gb300 import binding, build

pytestmark = pytest.mark.gpu
NEG = float("-inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


class Step:
    """Random codes and scales in pages scattered over a pool, NaN scales in the
    slots that no sequence owns."""

    def __init__(self, lens, n_new, H, Hk, d, page, seed, bound=0):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lens, self.n, self.H, self.Hk, self.d, self.page = list(lens), n_new, H, Hk, d, page
        self.max_len = max(*lens, bound, 1)
        pages = [-(-n // page) for n in lens]
        pool = sum(pages) + 2
        order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
        self.table = torch.full((len(lens), -(-self.max_len // page)), -7, dtype=torch.int32, device="cuda")
        rand = lambda *s: torch.rand(*s, device="cuda", generator=g)  # noqa: E731
        randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.codes = torch.randint(0, 256, (2, pool, Hk, page, d // 2), dtype=torch.uint8, device="cuda", generator=g)
        s = 0.05 + 0.1 * rand(2, pool, Hk, page, d // 64)
        self.scales = torch.stack((s, 0.3 * randn(*s.shape) - 7.5 * s), -1).to(torch.bfloat16)
        owned = torch.zeros(pool * page, dtype=torch.bool, device="cuda")
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
            page_of, slot = self.place(b)
            owned[page_of * page + slot] = True
        self.scales.masked_fill_(~owned.view(1, pool, 1, page, 1, 1), float("nan"))
        self.q = randn(len(lens), n_new, H, d).to(torch.bfloat16)
        self.scale = d ** -0.5

    def place(self, b):
        import torch
        t = torch.arange(self.lens[b], device="cuda")
        return self.table[b].long()[t // self.page], t % self.page

    def run(self):
        import torch
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        o, lse = binding.attention_decode_paged_q4(self.q, self.codes[0], self.scales[0], self.codes[1], self.scales[1],
                                                   self.table, lens, self.max_len, self.scale)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        return o, lse

    def held(self, i, b):
        """z and s of every element of sequence b's rows, and their codes: [L, Hk, d] each."""
        import torch
        page, slot = self.place(b)
        byte = self.codes[i][page, :, slot]
        sz = self.scales[i][page, :, slot].double().repeat_interleave(64, -2)
        return sz[..., 1], sz[..., 0], torch.stack((byte & 15, byte >> 4), -1).flatten(-2).double()

    def check(self, o, lse):
        import torch
        n, Hk, G, d = self.n, self.Hk, self.H // self.Hk, self.d
        for b, L in enumerate(self.lens):
            got, gl = o[b].double().view(n, Hk, G, d), lse[b].double().view(n, Hk, G)
            q = self.q[b].double().view(n, Hk, G, d)
            (kz, ks, kc), (vz, vs, vc) = self.held(0, b), self.held(1, b)
            last = L - n + torch.arange(n, device="cuda")
            hidden = (torch.arange(L, device="cuda") > last[:, None])[:, None, None]  # [n, 1, 1, L]
            none = last < 0
            assert not got[none].any() and bool((gl[none] == NEG).all())
            if L == 0 or bool(none.all()):
                continue
            x = (torch.einsum("nkgd,lkd->nkgl", q, kz + ks * kc) * self.scale).masked_fill(hidden, NEG)[~none]
            M = (torch.einsum("nkgd,lkd->nkgl", q.abs(), kz.abs() + ks * kc) * self.scale).masked_fill(hidden, 0.0)[~none]
            M, ref = M.amax(-1), torch.logsumexp(x, -1)
            p = torch.exp(x - ref[..., None])
            E = d * 2.0 ** -23 * M + 2.0 ** -22 + 2.0 ** -22 * M
            assert float(E.max()) < 0.05
            O, W = (torch.einsum("nkgl,lkd->nkgd", p, v) for v in (vz + vs * vc, vz.abs() + vs * vc))
            S = torch.stack([(p * vs[:, :, c].t()[None, :, None]).amax(-1) for c in range(0, d, 64)], -1)
            tol = 2.0 ** -8 * O.abs() + (4 * E[..., None] + 2.0 ** -11 + 2.0 ** -23 * (L / 32 + 64)) * W + \
                L * 2.0 ** -30 * S.repeat_interleave(64, -1)
            off = (got[~none] - O).abs()
            assert bool((off <= tol).all()), (b, float((off / tol).nan_to_num(1e9).max()))
            assert bool(((gl[~none] - ref).abs() <= E + 2.0 ** -24 * (L / 32 + 64) + 2.0 ** -22 * (1 + ref.abs())).all())


@pytest.mark.parametrize("r", [20, 26, 34, 40])
@pytest.mark.parametrize("n", [1, 2, 4])  # 4, 8 and 16 rows of a key head
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hk", [([3000, 700], 2), ([20000], 8)])  # a cluster for each item; even shares
def test_values_of_different_size_within_a_sequence(lens, Hk, d, n, r):
    """Every other tile's values are 2^r times larger, and its logits so far
    below the rest's that they have no weight (60 to 90 of them base 2): what
    they leave behind must not cost the other tiles' values their bits."""
    import torch
    x = Step(lens, n, 4 * Hk, Hk, d, 64, 8800 + d + n + r)
    x.q[..., :64] = x.q[..., :64].abs()
    for b in range(len(lens)):
        page, slot = x.place(b)
        low = torch.arange(lens[b], device="cuda") // 128 % 2 == 0
        page, slot = page[low], slot[low]
        # 64 elements of mean sqrt(2 / pi) each: 51 times the step.
        x.scales[0][page, :, slot, 0, 1] -= (r / 2 + 50) * math.log(2) / (51 * x.scale)
        x.scales[1][page, :, slot] *= 2.0 ** r
    x.check(*x.run())


def test_values_that_grow_with_their_weights():
    """Tiles of ever larger logits (by 7 base 2 each) and values 2^5 or 2^7
    times smaller from one to the next: the power of two follows both ways."""
    import torch
    for fall in (5, 7):
        x = Step([2048] * 6, 2, 8, 2, 128, 64, 8890 + fall)
        x.q[..., :64] = x.q[..., :64].abs()
        for b in range(6):
            page, slot = x.place(b)
            tile = (torch.arange(2048, device="cuda") // 128)[:, None]
            x.scales[0][page, :, slot, 0, 1] += (7.0 * (tile - 15) * math.log(2) / (51 * x.scale)).to(torch.bfloat16)
            x.scales[1][page, :, slot] *= torch.exp2(float(fall) * (15 - tile))[..., None, None].to(torch.bfloat16)
        x.check(*x.run())


def test_the_longest_sequence():
    """2^31 - 1 tokens (pages of the same block over and over): every logit 0,
    so that the sums of a warp's keys are whole numbers, and every value 1. The
    block of the last page reads as NaN in the slot behind the last token."""
    import torch
    page, lens = 65536, [2 ** 31 - 1, 100]
    codes = torch.randint(0, 256, (2, 1, page, 32), dtype=torch.uint8, device="cuda")
    k_scales, v_scales = (torch.zeros(2, 1, page, 1, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    v_scales[..., 1] = 1.0
    k_scales[1, :, -1], v_scales[1, :, -1] = float("nan"), float("nan")
    table = torch.zeros(2, 2 ** 31 // page, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.randn(2, 1, 64, device="cuda").to(torch.bfloat16)
    o, lse = binding.attention_decode_paged_q4(q, codes, k_scales, codes, v_scales, table,
                                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 2 ** 31 - 1, 0.1)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    assert bool((o == 1).all())
    # The parts' sums in base 2, joined in fp32 over at most 608 CTAs.
    for b, L in enumerate(lens):
        ref = math.log(L)
        assert abs(float(lse[b]) - ref) <= 2.0 ** -21 * (1 + ref) + 608 * 2.0 ** -24


@pytest.mark.parametrize("d,n,H", [(64, 1, 8), (64, 3, 24), (128, 1, 32), (128, 5, 24)])
def test_runs_of_many_tiles(d, n, H):
    """Ragged sequences, empty ones among them, of enough tiles that an item
    counts as some tiles more in the shares: runs that begin and end anywhere,
    before the first tile of an item too, whole items between them."""
    import random
    rng = random.Random(d + n)
    lens = [rng.choice([0, rng.randint(1, 300), rng.randint(1000, 9000), rng.randint(5000, 9000)]) for _ in range(96)]
    x = Step(lens, n, H, 8, d, 64, 8950 + d + n, bound=20000)
    ctas = 152 * ((4 if d == 64 else 3) - (n * H // 8 > 8))
    assert sum(-(-L // 128) for L in lens) * 8 >= 8 * ctas
    o, lse = x.run()
    x.check(o, lse)
    again = x.run()
    assert bool((o == again[0]).all()) and bool((lse == again[1]).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("bound", [0, 20000])
def test_logits_past_fp32(d, n, bound):
    """Where every logit overflows to -inf, O is 0 and the LSE -inf; where one
    is +inf, both are NaN; the other sequence keeps its bits."""
    import torch
    x = Step([500, 300], n, 8, 2, d, 64, 8990 + d + n, bound=bound)
    o, lse = x.run()
    page, slot = x.place(0)
    x.q[0] = x.q[0].abs() * 2.0 ** 40
    x.q[0, :, ::2] *= -1
    for count in (500, 128):  # the keys whose minimum lies far below zero: all of them, the first tile's
        if count < 500:
            x.scales[0][page, :, slot, :, 1] = 0.0
        x.scales[0][page[:count], :, slot[:count], :, 1] = -2.0 ** 125
        o1, l1 = x.run()
        assert torch.equal(o1[1], o[1]) and torch.equal(l1[1], lse[1])
        assert bool(o1[0, :, ::2].isnan().all()) and bool(l1[0, :, ::2].isnan().all())
        if count == 500:
            assert not o1[0, :, 1::2].any() and bool((l1[0, :, 1::2] == NEG).all())
        else:
            assert bool(o1[0, :, 1::2].isfinite().all()) and bool(l1[0, :, 1::2].isfinite().all())
