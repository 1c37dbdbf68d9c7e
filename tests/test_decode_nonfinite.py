"""Non-finite values among the visible inputs of a shared-prefix decoding step
(fa_decode_shared_prefix): a logit of NaN or +inf makes the whole row of O and
its LSE NaN, as the definition does; a logit of -inf has no weight; a NaN in V
makes its column of O NaN and leaves the LSE alone. O = 0 with LSE = -inf means
"no keys" and nothing else. Rows that do not see the value keep their bits.
Both routes of the prefix (streamed, and in 128-row tiles), rows with one part
and with many."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build
from test_decode_shared import Step

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
H, HK = 8, 2
G = H // HK

# (sequences of each prefix, prefix lengths, own lengths)
STEPS = {
    "streamed, several parts": ([3, 1], [900, 300], [200, 0, 64, 1]),
    "streamed, one part": ([2], [60], [0, 0]),
    "own tokens alone": ([0], [0], [50, 300]),
    "tiles, several parts": ([40], [900], [i % 3 for i in range(40)]),
    "tiles, one part": ([8], [100], [0] * 8),
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def step(name, d):
    return Step(*STEPS[name], H, HK, d, 64, 8800 + d)


def run(x):
    import torch
    o, lse = binding.attention_decode_shared_prefix(*x.args())
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    return o, lse


def a_key(x, last):
    """(block, slot) of a visible key, the first or last of prefix 0 (of
    sequence 1 where there is no prefix), and the sequences that see it."""
    if x.plens[0]:
        row, n, seqs = x.ptab[0], int(x.plens[0]), range(int(x.cu[0]), int(x.cu[1]))
    else:
        row, n, seqs = x.stab[1], int(x.slens[1]), [1]
    t = n - 1 if last else 0
    return int(row[t // x.page]), t % x.page, list(seqs)


def same_elsewhere(got, want, hit):
    """hit: bool [B, H]; the other rows keep their bits."""
    import torch
    keep = torch.from_numpy(~hit).cuda()
    assert torch.equal(got[0][keep].view(torch.int16), want[0][keep].view(torch.int16))
    assert torch.equal(got[1][keep], want[1][keep])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", STEPS)
def test_a_query_of_nan(name, d):
    import torch
    x = step(name, d)
    want = run(x)
    x.q[1, 3, 5] = NAN
    o, lse = run(x)
    hit = np.zeros((x.B, H), bool)
    hit[1, 3] = True
    assert bool(torch.isnan(o[1, 3]).all()) and bool(torch.isnan(lse[1, 3]))
    same_elsewhere((o, lse), want, hit)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("name", STEPS)
def test_a_visible_key_of_nan(name, last, d):
    import torch
    x = step(name, d)
    want = run(x)
    blk, slot, seqs = a_key(x, last)
    x.k[blk, slot, 1, d - 1] = NAN
    o, lse = run(x)
    hit = np.zeros((x.B, H), bool)
    hit[seqs, G:] = True  # the heads of key head 1
    rows = torch.from_numpy(hit).cuda()
    assert bool(torch.isnan(o[rows]).all()) and bool(torch.isnan(lse[rows]).all())
    same_elsewhere((o, lse), want, hit)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("name", STEPS)
def test_a_visible_value_of_nan(name, last, d):
    import torch
    x = step(name, d)
    want = run(x)
    blk, slot, seqs = a_key(x, last)
    x.v[blk, slot, 1, 7] = NAN
    o, lse = run(x)
    hit = np.zeros((x.B, H), bool)
    hit[seqs, G:] = True
    rows = torch.from_numpy(hit).cuda()
    assert bool(torch.isnan(o[rows][:, 7]).all())
    assert torch.equal(lse, want[1])
    same_elsewhere((o, lse), want, hit)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", STEPS)
def test_a_visible_key_of_infinity(name, d):
    """Rows whose query is positive there have a logit of +inf (NaN by the
    definition: inf - inf), the others one of -inf: that key weighs nothing,
    and what is left is the step without it."""
    import torch
    x = step(name, d)
    blk, slot, seqs = a_key(x, True)
    x.k[blk, slot, 1, 2] = INF
    up = np.zeros((x.B, H), bool)
    up[seqs, G:] = (x.q[seqs, G:, 2] > 0).cpu().numpy()
    assert up.any()
    o, lse = run(x)
    rows = torch.from_numpy(up).cuda()
    assert bool(torch.isnan(o[rows]).all()) and bool(torch.isnan(lse[rows]).all())
    lens = x.plens if x.plens[0] else x.slens
    lens[0 if x.plens[0] else 1] -= 1
    ro, rl, ra = x.oracle()
    go, gl = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    down = np.zeros((x.B, H), bool)
    down[seqs, G:] = ~up[seqs, G:]
    assert np.all(np.abs(go[down] - ro[down]) <= 2.0 ** -8 * np.abs(ro[down]) + 2.0 ** -10 * ra[down])
    assert np.all(np.abs(gl[down] - rl[down]) <= 2.0 ** -11)
