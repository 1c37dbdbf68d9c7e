"""Prompt attention with grouped heads (fa_fwd_varlen_gqa, fa_bwd_varlen_gqa)
against the fp64 oracle, whose key heads are repeated for every query head of
their group and whose dK, dV are summed over it. The forward is also compared
bit for bit with fa_fwd_varlen on repeated key heads: each row goes through
the same key blocks with the same arithmetic, whatever tile it sits in."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build, synth
import parity_util as pu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def cum(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Packed:
    def __init__(self, lens_q, lens_k, H, Hk, d, seed, spare=0):
        import torch
        self.cu_q, self.cu_k = cum(lens_q), cum(lens_k)
        self.H, self.Hk, self.d = H, Hk, d
        tq, tk = int(self.cu_q[-1]) + spare, int(self.cu_k[-1]) + spare
        bits = {"q": synth.bf16_normal_tensor(seed, synth.STREAM_Q, (tq, H, d)),
                "k": synth.bf16_normal_tensor(seed, synth.STREAM_K, (tk, Hk, d)),
                "v": synth.bf16_normal_tensor(seed, synth.STREAM_V, (tk, Hk, d)),
                "do": synth.bf16_normal_tensor(seed, synth.STREAM_DO, (tq, H, d))}
        self.dev = {n: pu.to_device(b) for n, b in bits.items()}
        self.f = {n: synth.bf16_bits_to_f64(b) for n, b in bits.items()}
        self.cu = torch.from_numpy(self.cu_q).cuda(), torch.from_numpy(self.cu_k).cuda()
        self.max_q, self.max_k = max(max(lens_q), 1), max(max(lens_k), 1)
        self.scale = 1 / np.sqrt(d)

    def args(self, causal):
        return (*self.cu, self.max_q, self.max_k, self.scale, causal)

    def qkv(self):
        return self.dev["q"], self.dev["k"], self.dev["v"]

    def repeated(self, name):
        return np.repeat(self.f[name], self.H // self.Hk, axis=1)

    def grouped(self, g):
        """Gradients of repeated key heads summed over each group."""
        return g.reshape(g.shape[0], self.Hk, self.H // self.Hk, self.d).sum(2)


CASES = [
    # (H, Hk, lens_q, lens_k)
    (8, 2, [300, 1, 129, 0, 128], [300, 1, 129, 0, 128]),  # four heads a tile; tile edges, empty, single
    (6, 2, [17, 250, 64], [400, 250, 700]),                # three heads a tile: 126 of its rows
    (7, 1, [300, 5, 200], [100, 5, 31]),                   # seven; more queries than keys: empty rows
    (5, 5, [1, 1, 140, 1], [513, 90, 1, 260]),             # full heads
    (16, 1, [70, 0, 9], [70, 40, 300]),                    # sixteen heads a tile; a sequence without queries
    (24, 1, [33, 12], [33, 0]),                            # eight a tile (24 would waste rows); no keys
    (44, 4, [31, 3], [90, 3]),                             # eleven: one head a tile
    (2, 1, [1000], [1500]),                                # continued prompt over many blocks
    (16, 8, [100 + 9 * i for i in range(20)], [100 + 9 * i for i in range(20)]),  # more key blocks than SMs
    (64, 1, [5, 130], [40, 130]),                          # 64 heads a tile: two tokens
    (256, 2, [3, 1, 9], [3, 70, 9]),                       # 128 heads a tile: one token
    (4, 1, [700, 650], [700, 650]),                        # few key blocks: their pairs shared out over CTAs
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_against_oracle(d, causal, case):
    import torch
    H, Hk, lq, lk = CASES[case]
    x = Packed(lq, lk, H, Hk, d, 7100 + 17 * case + d)
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(causal))
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    ro, rl = oracle.varlen_forward(x.f["q"], x.repeated("k"), x.repeated("v"), x.cu_q, x.cu_k, x.scale, causal)
    go = pu.bf16_tensor_to_f64(o)
    assert np.all(np.isfinite(go))
    assert pu.o_err(go, ro) <= pu.O_ATOL
    assert pu.max_abs(lse.cpu().numpy(), rl) <= pu.LSE_ATOL


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,d,causal", [(8, 2, 128, True), (6, 2, 64, True), (12, 1, 128, False), (7, 7, 64, True)])
def test_forward_equals_repeated_key_heads_bit_for_bit(H, Hk, d, causal):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    lens = [3000, 1, 257, 900, 64]
    cu = torch.from_numpy(cum(lens)).cuda()
    T = sum(lens)
    q = 2 * torch.randn(T, H, d, device="cuda", generator=g)
    q, k, v = (t.to(torch.bfloat16) for t in (q, *torch.randn(2, T, Hk, d, device="cuda", generator=g)))
    o, lse = binding.attention_forward_varlen_gqa(q, k, v, cu, cu, 3000, 3000, d ** -0.5, causal)
    kr, vr = (t.repeat_interleave(H // Hk, dim=1) for t in (k, v))
    ro, rl = binding.attention_forward_varlen(q, kr, vr, cu, cu, 3000, 3000, d ** -0.5, causal)
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), ro.view(torch.int16))
    assert torch.equal(lse, rl)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,d,causal,lens,extra", [
    (16, 4, 128, True, [3000] + [50 + i for i in range(40)], 0),          # several passes over 32 sequences
    (6, 2, 64, False, [0, 0, 1, 2600, 0, 300, 77, 1], 0),
    (8, 8, 64, True, [7, 1500, 0, 63, 64, 65], 40),                       # more keys than queries, full heads
    (4, 1, 128, True, [1 + 13 * i % 61 for i in range(300)] + [2000], 0),
    (8, 1, 128, True, [20000, 30000, 9, 100, 26000, 5, 900, 40000], 0),   # K and V of the batch past half the L2
])
def test_short_prompts_beside_long_ones(H, Hk, d, causal, lens, extra):
    """Batches whose grid holds only the tiles that exist: every row as with
    repeated key heads, bit for bit, and the same again when the longest
    length named is larger than the batch's."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(43)
    lens_k = [n + extra for n in lens]
    cq, ck = (torch.from_numpy(cum(n)).cuda() for n in (lens, lens_k))
    T, Tk = sum(lens), sum(lens_k)
    q = torch.randn(T, H, d, device="cuda", generator=g).to(torch.bfloat16)
    k, v = (torch.randn(Tk, Hk, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    kr, vr = (t.repeat_interleave(H // Hk, dim=1) for t in (k, v))
    ro, rl = binding.attention_forward_varlen(q, kr, vr, cq, ck, max(lens), max(lens_k), d ** -0.5, causal)
    for longest in (max(lens), min(5 * max(lens), T)):
        o = torch.full_like(q, float("nan"))
        lse = torch.full((H, T), float("nan"), device="cuda")
        binding.fa_fwd_varlen_gqa(q, k, v, o, lse, cq, ck, longest, max(lens_k), d ** -0.5, causal)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        assert torch.equal(o.view(torch.int16), ro.view(torch.int16))
        assert torch.equal(lse, rl)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_backward_against_oracle(d, causal, deterministic, case):
    import torch
    H, Hk, lq, lk = CASES[case]
    x = Packed(lq, lk, H, Hk, d, 7300 + 19 * case + d)
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(causal))
    got = binding.attention_backward_varlen_gqa(*x.qkv(), o, lse, x.dev["do"], *x.args(causal),
                                                deterministic=deterministic)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    rq, rk, rv = oracle.varlen_backward(x.f["q"], x.repeated("k"), x.repeated("v"), x.f["do"], x.cu_q, x.cu_k,
                                        x.scale, causal)
    for name, g, r in (("dQ", got[0], rq), ("dK", got[1], x.grouped(rk)), ("dV", got[2], x.grouped(rv))):
        g = pu.bf16_tensor_to_f64(g)
        assert np.all(np.isfinite(g)), name
        err = pu.max_abs(g, r) / max(float(np.max(np.abs(r))), pu.ZERO_REF_FLOOR)
        assert err <= pu.GRAD_RTOL, (name, err)
    if deterministic:
        again = binding.attention_backward_varlen_gqa(*x.qkv(), o, lse, x.dev["do"], *x.args(causal),
                                                      deterministic=True)
        for a, b in zip(got, again):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.gpu
def test_gradients_match_differences():
    """dK and dV of shared heads against central differences of the fp64
    forward of one packed sequence, along seeded directions. The kernel's
    gradients are within 1e-2 of max |gradient| per element (as above); along
    a unit direction over n elements that is at most 1e-2 * max * sqrt(n)."""
    import torch
    H, Hk, d, L = 6, 2, 64, 40
    x = Packed([L], [L + 9], H, Hk, d, 7500)
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(True))
    _, dk, dv = binding.attention_backward_varlen_gqa(*x.qkv(), o, lse, x.dev["do"], *x.args(True))
    torch.cuda.synchronize()

    def loss(k, v):
        r = lambda t: np.repeat(t, H // Hk, axis=1)  # noqa: E731
        return float(np.sum(oracle.varlen_forward(x.f["q"], r(k), r(v), x.cu_q, x.cu_k, x.scale, True)[0] * x.f["do"]))

    rng = np.random.default_rng(3)
    for which, g in (("k", dk), ("v", dv)):
        g = pu.bf16_tensor_to_f64(g)
        u = rng.standard_normal(g.shape)
        u /= np.linalg.norm(u)
        h = 1e-4
        kv = lambda s: (x.f["k"] + (s * h * u if which == "k" else 0), x.f["v"] + (s * h * u if which == "v" else 0))  # noqa: E731
        diff = (loss(*kv(1)) - loss(*kv(-1))) / (2 * h)
        assert abs(diff - float(np.sum(g * u))) <= 1e-2 * np.max(np.abs(g)) * np.sqrt(g.size) + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,d", [(8, 2, 128), (6, 2, 64)])
def test_rows_of_no_sequence_stay_as_they_were(H, Hk, d):
    """Rows behind the last sequence hold NaN in every input: they must reach
    no output, and their own output rows keep what was in them."""
    import torch
    lens, spare = [130, 7, 60], 50
    x = Packed(lens, lens, H, Hk, d, 7600, spare=spare)
    T = sum(lens)
    clean = Packed(lens, lens, H, Hk, d, 7600)
    for n in ("q", "k", "v", "do"):
        clean.dev[n] = x.dev[n][:T].clone()
        x.dev[n][T:] = float("nan")
    o, dq, dk, dv = (torch.full_like(x.dev[n], 7.0) for n in ("q", "q", "k", "v"))
    lse = torch.full((H, T + spare), 7.0, device="cuda")
    binding.fa_fwd_varlen_gqa(*x.qkv(), o, lse, *x.args(True))
    binding.fa_bwd_varlen_gqa_deterministic(*x.qkv(), o, lse, x.dev["do"], dq, dk, dv, *x.args(True))
    ro, rl = binding.attention_forward_varlen_gqa(*clean.qkv(), *clean.args(True))
    rg = binding.attention_backward_varlen_gqa(*clean.qkv(), ro, rl, clean.dev["do"], *clean.args(True),
                                               deterministic=True)
    torch.cuda.synchronize()
    for t, r in zip((o, dq, dk, dv), (ro, *rg)):
        assert torch.equal(t[:T], r) and bool((t[T:] == 7).all())
    assert torch.equal(lse[:, :T], rl) and bool((lse[:, T:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,d,lq,lk", [
    (8, 2, 128, [6000, 1, 0, 2200, 129, 700, 4100, 128], [6000, 1, 90, 2500, 129, 600, 4100, 0]),
    (12, 12, 64, [2000, 30, 1500, 900, 1999], [2000, 30, 1500, 900, 1999]),
    (16, 4, 128, [900 - 40 * i for i in range(20)], [900 - 40 * i for i in range(20)]),
])
def test_backward_orders_take_every_key_block_once(H, Hk, d, lq, lk):
    """The default order starts heavy key blocks first and keeps light ones
    back, the deterministic one counts them off plainly. Each key block's dK
    and dV sum over the same pairs in the same order in both, bit for bit; dQ
    sums over key blocks in another order: two bf16 roundings of nearly equal
    values, at most 2^-8 of the largest apart. No row stays unwritten."""
    import torch
    x = Packed(lq, lk, H, Hk, d, 7700)
    o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(True))
    out = []
    for f in (binding.fa_bwd_varlen_gqa, binding.fa_bwd_varlen_gqa_deterministic):
        g = [torch.full_like(x.dev[n], float("nan")) for n in ("q", "k", "v")]
        f(*x.qkv(), o, lse, x.dev["do"], *g, *x.args(True))
        out.append(g)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    (dq, dk, dv), (rq, rk, rv) = out
    assert torch.equal(dk.view(torch.int16), rk.view(torch.int16))
    assert torch.equal(dv.view(torch.int16), rv.view(torch.int16))
    assert bool(torch.isfinite(dq).all()) and bool(torch.isfinite(dk).all())
    assert float((dq.float() - rq.float()).abs().max()) <= 1e-2 * float(rq.float().abs().max())


@pytest.mark.gpu
def test_values_outside_f16_take_the_second_pass():
    """A V beyond f16's range makes its tiles run again in bf16, grouped tiles
    (126 of 128 rows in use) among them. O is linear in V: 1e-2 * scale of V."""
    import torch
    for mul in (2.0 ** 20, 2.0 ** -30):
        x = Packed([200, 33], [200, 90], 6, 2, 128, 7700)
        v = (x.dev["v"].float() * mul).to(torch.bfloat16)
        o, lse = binding.attention_forward_varlen_gqa(x.dev["q"], x.dev["k"], v, *x.args(True))
        torch.cuda.synchronize()
        ro, rl = oracle.varlen_forward(x.f["q"], x.repeated("k"), x.repeated("v"), x.cu_q, x.cu_k, x.scale, True)
        assert pu.o_err(pu.bf16_tensor_to_f64(o) / mul, ro) <= pu.O_ATOL
        assert pu.max_abs(lse.cpu().numpy(), rl) <= pu.LSE_ATOL


@pytest.mark.gpu
def test_captured_and_on_two_streams():
    """A captured forward + backward replayed on new inputs, with an eager call
    of another problem under way on a second stream with its own workspace,
    equals the same calls made alone (deterministic order: bit for bit)."""
    import torch
    xs = [Packed([300, 20, 513], [300, 20, 513], 8, 2, 128, 7800 + i) for i in range(2)]
    other = Packed([700, 90], [700, 90], 6, 2, 64, 7900)

    def alone(x):
        o, lse = binding.attention_forward_varlen_gqa(*x.qkv(), *x.args(True))
        return (o, lse, *binding.attention_backward_varlen_gqa(*x.qkv(), o, lse, x.dev["do"], *x.args(True),
                                                               deterministic=True))

    want, want_other = [alone(x) for x in xs], alone(other)
    bufs = {n: xs[0].dev[n].clone() for n in ("q", "k", "v", "do")}
    out = [torch.empty_like(t) for t in want[0]]
    ws = torch.empty(binding.fa_bwd_workspace_size(3, 8, 513, 128), dtype=torch.uint8, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()

    def step(stream):
        qkv = bufs["q"], bufs["k"], bufs["v"]
        binding.fa_fwd_varlen_gqa(*qkv, out[0], out[1], *xs[0].args(True), stream)
        binding.fa_bwd_varlen_gqa_deterministic(*qkv, out[0], out[1], bufs["do"], *out[2:], *xs[0].args(True), ws,
                                                stream)

    torch.cuda.synchronize()
    step(s1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        step(s1)
    for x, w in zip(xs, want):
        for n in bufs:
            bufs[n].copy_(x.dev[n])
        torch.cuda.synchronize()
        with torch.cuda.stream(s2):
            got_other = alone(other)
        with torch.cuda.stream(s1):
            graph.replay()
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        for a, b in zip((*out, *got_other), (*w, *want_other)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_tensors_past_2_31_elements():
    """A packed batch of 2.2e9 query elements: sequences at its boundaries and at
    its end give, bit for bit, what they give in a small batch (forward and
    deterministic backward)."""
    import torch
    H, Hk, d, L, B = 32, 4, 128, 1000, 540
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    T = B * L
    make = lambda h: torch.randn(L, h, d, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    src = {n: [make(h) for _ in range(3)] for n, h in (("q", H), ("k", Hk), ("v", Hk), ("do", H))}
    full = {n: torch.cat([s[b % 3] for b in range(B)]) for n, s in src.items()}
    assert full["q"].numel() > 2 ** 31
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * L
    args = (cu, cu, L, L, d ** -0.5, True)
    o, lse = binding.attention_forward_varlen_gqa(full["q"], full["k"], full["v"], *args)
    grads = binding.attention_backward_varlen_gqa(full["q"], full["k"], full["v"], o, lse, full["do"], *args,
                                                  deterministic=True)
    # The same sequences in a batch of twenty: as many key blocks per head as
    # keep it from sharing them out over clusters (which add up in another order).
    n = 20
    few = {x: torch.cat([t[b % 3] for b in range(n)]) for x, t in src.items()}
    cf = cu[:n + 1].contiguous()
    af = (cf, cf, L, L, d ** -0.5, True)
    fo, fl = binding.attention_forward_varlen_gqa(few["q"], few["k"], few["v"], *af)
    fg = binding.attention_backward_varlen_gqa(few["q"], few["k"], few["v"], fo, fl, few["do"], *af,
                                               deterministic=True)
    torch.cuda.synchronize()
    for b in (B - 1, B - 2, 2 ** 30 // (L * H * d), 2 ** 31 // (L * H * d), 0):
        rows, same = slice(b * L, (b + 1) * L), slice(b % 3 * L, (b % 3 + 1) * L)
        assert torch.equal(o[rows], fo[same]) and torch.equal(lse[:, rows], fl[:, same])
        for t, r in zip(grads, fg):
            assert torch.equal(t[rows], r[same])


FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced (rejected first)
SIZES = dict(batch=2, H=8, Hk=2, d=64, tq=40, tk=40, mq=30, mk=30, scale=0.125)


@pytest.mark.parametrize("change,expect", [
    (dict(Hk=3), binding.FA_ERR_INVALID),
    (dict(Hk=0), binding.FA_ERR_INVALID),
    (dict(Hk=16), binding.FA_ERR_INVALID),
    (dict(batch=0), binding.FA_ERR_INVALID),
    (dict(mq=41), binding.FA_ERR_INVALID),
    (dict(mk=0), binding.FA_ERR_INVALID),
    (dict(scale=float("inf")), binding.FA_ERR_INVALID),
    (dict(d=80), binding.FA_ERR_UNSUPPORTED),
    (dict(ptr=FAKE + 8), binding.FA_ERR_UNSUPPORTED),
    (dict(ptr=None), binding.FA_ERR_INVALID),
])
def test_refusals(change, expect):
    lib = binding.load_library()
    a = {**SIZES, "ptr": FAKE, **change}
    sizes = (a["batch"], a["H"], a["Hk"], a["d"], a["tq"], a["tk"], a["mq"], a["mk"], a["scale"], 1)
    assert lib.fa_fwd_varlen_gqa(a["ptr"], *([FAKE] * 6), *sizes, None) == expect
    for fn in (lib.fa_bwd_varlen_gqa, lib.fa_bwd_varlen_gqa_deterministic):
        assert fn(a["ptr"], *([FAKE] * 10), *sizes, FAKE, 1 << 40, None) == expect


def test_backward_refuses_a_small_workspace():
    lib = binding.load_library()
    a = SIZES
    sizes = (a["batch"], a["H"], a["Hk"], a["d"], a["tq"], a["tk"], a["mq"], a["mk"], a["scale"], 1)
    need = lib.fa_bwd_workspace_size(2, 8, 30, 64)
    assert lib.fa_bwd_varlen_gqa(*([FAKE] * 11), *sizes, FAKE, need - 1, None) == binding.FA_ERR_WORKSPACE
    assert lib.fa_bwd_varlen_gqa(*([FAKE] * 11), *sizes, None, need, None) == binding.FA_ERR_WORKSPACE
