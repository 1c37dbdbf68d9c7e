"""Non-finite values in a paged decoding step (fa_decode_paged): NaN in slots of
an owned page that its sequence has not written reaches nothing; a NaN or +inf
logit of a visible key makes the row's O and LSE NaN (O = 0 with LSE = -inf
means no keys); rows that do not see it keep their bits. Rows of one split and
of several."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


class Step:
    def __init__(self, lens, H, d, page):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(23)
        B, width = len(lens), -(-max(lens) // page)
        self.lens, self.page, self.d, self.max_len = lens, page, d, max(lens)
        self.q = torch.randn(B, H, d, device="cuda", generator=g).to(torch.bfloat16)
        self.k, self.v = (torch.randn(B * width, page, H, d, device="cuda", generator=g).to(torch.bfloat16)
                          for _ in range(2))
        self.table = torch.randperm(B * width, device="cuda", generator=g).to(torch.int32).view(B, width)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def run(self):
        import torch
        o, lse = binding.attention_decode_paged(self.q, self.k, self.v, self.table, self.seq_lens, self.max_len,
                                                self.d ** -0.5)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        return o, lse

    def at(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page


# (own lengths, heads): 1024 items or so in all, so many heads keep a row in one split.
STEPS = [([700, 0, 65, 64, 1], 3), ([130, 100, 1, 64], 300)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", range(len(STEPS)))
def test_slots_that_no_token_has_written(step, d):
    import torch
    x = Step(*STEPS[step], d, 128)
    want = x.run()
    for b, n in enumerate(x.lens):
        for t in range(n, x.table.shape[1] * x.page):
            blk, slot = x.at(b, t)
            x.k[blk, slot] = x.v[blk, slot] = NAN
    o, lse = x.run()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["query", "first key", "last key", "infinite logit"])
@pytest.mark.parametrize("step", range(len(STEPS)))
def test_a_logit_that_is_not_finite(step, what, d):
    import torch
    x = Step(*STEPS[step], d, 128)
    want = x.run()
    if what == "query":
        x.q[0, 1, 5] = NAN
    elif what == "infinite logit":
        blk, slot = x.at(0, 10)
        x.k[blk, slot, 1, 5] = float("inf") if float(x.q[0, 1, 5]) > 0 else -float("inf")
    else:
        blk, slot = x.at(0, 0 if what == "first key" else x.lens[0] - 1)
        x.k[blk, slot, 1, d - 1] = NAN
    o, lse = x.run()
    assert bool(torch.isnan(o[0, 1]).all()) and bool(torch.isnan(lse[0, 1]))
    keep = torch.ones(x.q.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
