"""The grouped-head operators as a model uses them, one after the other: fused
projections -> norm + rotation -> prompt attention -> pages of a cache ->
decoding steps that share the prompts; and the training pass back through both
operators into the fused projections' gradient. Each stage is compared with
the fp64 oracle on what the stage before handed over, with the tolerances of
its own tests. Also: the bounded waits of the kernels, and that the entry
points allocate nothing."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build, synth
import parity_util as pu

pytestmark = pytest.mark.gpu
H, HK, D, PAGE = 8, 2, 128, 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


class Model:
    """Weights, tables and fused projections [T, (H + 2 HK) D] of a step's tokens."""

    def __init__(self, seed):
        import torch
        rng = np.random.default_rng(seed)
        self.seed, self.n = seed, 0
        freq = 10000.0 ** (-np.arange(0, D, 2) / D)
        angle = np.arange(2000)[:, None] * freq
        self.tab = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        self.cos, self.sin = (torch.from_numpy(t).cuda() for t in self.tab)
        self.w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to(torch.bfloat16).cuda()
                  for _ in range(2)]
        self.scale = D ** -0.5

    def project(self, positions):
        """(q, k, v views of a fused tensor, positions on the device) of new tokens."""
        import torch
        self.n += 1
        T = len(positions)
        qkv = pu.to_device(synth.bf16_normal_tensor(self.seed + 7919 * self.n, synth.STREAM_Q, (T, (H + 2 * HK) * D)))
        q, k, v = qkv[:, :H * D], qkv[:, H * D:(H + HK) * D], qkv[:, (H + HK) * D:]
        return (q.view(T, H, D), k.view(T, HK, D), v.view(T, HK, D),
                torch.from_numpy(np.asarray(positions, np.int32)).cuda())

    def rotate(self, q, k, pos):
        """The operator's q and k, checked."""
        out = binding.qk_norm_rope(q, k, *self.w, self.cos, self.sin, pos)
        for x, w, y in zip((q, k), self.w, out):
            x, w = pu.bf16_tensor_to_f64(x), pu.bf16_tensor_to_f64(w)
            p = pos.cpu().numpy()
            ref = oracle.norm_rope_forward(x, w, *self.tab, p, 1e-6, False)
            both = np.abs(oracle.norm_rope_forward(x, w, self.tab[0], 0 * self.tab[1], p, 1e-6, False)) + \
                np.abs(oracle.norm_rope_forward(x, w, 0 * self.tab[0], self.tab[1], p, 1e-6, False))
            assert np.all(np.abs(pu.bf16_tensor_to_f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * both)
        return out


def rep(x):
    return np.repeat(pu.bf16_tensor_to_f64(x), H // HK, axis=1)


def test_prompts_then_shared_decoding():
    import torch
    m = Model(8100)
    lens = [200, 77]             # two prompts
    answers = [3, 2]             # sampled for each
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    q, k, v, pos = m.project(np.concatenate([np.arange(n) for n in lens]))
    q, k = m.rotate(q, k, pos)
    v = v.contiguous()
    o, lse = binding.attention_forward_varlen_gqa(q, k, v, cu, cu, max(lens), max(lens), m.scale, True)
    c = cu.cpu().numpy()
    ro, rl = oracle.varlen_forward(pu.bf16_tensor_to_f64(q), rep(k), rep(v), c, c, m.scale, True)
    assert pu.o_err(pu.bf16_tensor_to_f64(o), ro) <= pu.O_ATOL
    assert pu.max_abs(lse.cpu().numpy(), rl) <= pu.LSE_ATOL

    # The prompts' keys and values go into pages, the answers start empty.
    B, steps = sum(answers), 3
    owner = np.repeat(np.arange(2), answers)
    pages = [-(-n // PAGE) for n in lens]
    pool = sum(pages) + B
    order = np.random.default_rng(1).permutation(pool).astype(np.int32)
    ptab = np.zeros((2, max(pages)), np.int32)
    kp, vp = (torch.full((pool, PAGE, HK, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = 0
    for p, n in enumerate(lens):
        ptab[p, :pages[p]] = order[at:at + pages[p]]
        slots = torch.from_numpy((order[at + np.arange(n) // PAGE].astype(np.int64) * PAGE + np.arange(n) % PAGE)).cuda()
        for cache, x in ((kp, k), (vp, v)):
            cache.view(-1, HK, D)[slots] = x[c[p]:c[p + 1]]
        at += pages[p]
    stab = order[at:].reshape(B, 1).copy()
    dev = [torch.from_numpy(x).cuda() for x in (ptab, np.asarray(lens, np.int32),
                                                np.concatenate([[0], np.cumsum(answers)]).astype(np.int32), stab)]
    hist = [(k[c[p]:c[p + 1]], v[c[p]:c[p + 1]]) for p in owner]
    for s in range(steps):
        q1, k1, v1, pos = m.project([lens[p] + s for p in owner])
        q1, k1 = m.rotate(q1, k1, pos)
        v1 = v1.contiguous()
        slots = torch.from_numpy(stab[:, 0].astype(np.int64) * PAGE + s).cuda()
        kp.view(-1, HK, D)[slots], vp.view(-1, HK, D)[slots] = k1, v1
        own = torch.full((B,), s + 1, dtype=torch.int32, device="cuda")
        o1, l1 = binding.attention_decode_shared_prefix(q1, kp, vp, *dev, own, max(answers), max(lens), steps, m.scale)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        # The same step as prompt attention: each sequence's one query over its
        # whole history (prompt and answer so far).
        hist = [(torch.cat((a, k1[b:b + 1])), torch.cat((x, v1[b:b + 1]))) for b, (a, x) in enumerate(hist)]
        kk, vv = (torch.cat([h[i] for h in hist]).contiguous() for i in range(2))
        cq = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        ck = torch.tensor(np.concatenate([[0], np.cumsum([len(h[0]) for h in hist])]), dtype=torch.int32, device="cuda")
        o2, l2 = binding.attention_forward_varlen_gqa(q1, kk, vv, cq, ck, 1, max(len(h[0]) for h in hist), m.scale, True)
        ro, rl = oracle.varlen_forward(pu.bf16_tensor_to_f64(q1), rep(kk), rep(vv), cq.cpu().numpy(), ck.cpu().numpy(),
                                       m.scale, True)
        for o, l in ((o1, l1.t()), (o2, l2)):
            assert pu.o_err(pu.bf16_tensor_to_f64(o), ro) <= pu.O_ATOL
            assert pu.max_abs(l.cpu().numpy(), rl) <= pu.LSE_ATOL


def test_training_pass_into_the_fused_gradient():
    import torch
    m = Model(8200)
    lens = [150, 1, 90]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    T = sum(lens)
    q0, k0, v0, pos = m.project(np.concatenate([np.arange(n) for n in lens]))
    q, k = m.rotate(q0, k0, pos)
    v = v0.contiguous()
    args = (cu, cu, max(lens), max(lens), m.scale, True)
    o, lse = binding.attention_forward_varlen_gqa(q, k, v, *args)
    do = pu.to_device(synth.bf16_normal_tensor(8201, synth.STREAM_DO, (T, H, D)))
    dq, dk, dv = binding.attention_backward_varlen_gqa(q, k, v, o, lse, do, *args)
    grad = torch.empty(T, (H + 2 * HK) * D, dtype=torch.bfloat16, device="cuda")
    gq, gk = grad[:, :H * D].view(T, H, D), grad[:, H * D:(H + HK) * D].view(T, HK, D)
    grad[:, (H + HK) * D:] = dv.view(T, HK * D)
    dw = [torch.empty(D, device="cuda") for _ in range(2)]
    binding.fa_qk_norm_rope_bwd(q0, k0, *m.w, m.cos, m.sin, pos, dq, dk, gq, gk, *dw)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    c = cu.cpu().numpy()
    rq, rk, rv = oracle.varlen_backward(pu.bf16_tensor_to_f64(q), rep(k), rep(v), pu.bf16_tensor_to_f64(do), c, c,
                                        m.scale, True)
    for got, ref in ((dq, rq), (dk, rk.reshape(T, HK, -1, D).sum(2)), (dv, rv.reshape(T, HK, -1, D).sum(2))):
        assert pu.max_abs(pu.bf16_tensor_to_f64(got), ref) <= pu.GRAD_RTOL * np.max(np.abs(ref))
    for x, w, g, dx, dwx in ((q0, m.w[0], dq, gq, dw[0]), (k0, m.w[1], dk, gk, dw[1])):
        rx, rw, mag = oracle.norm_rope_backward(pu.bf16_tensor_to_f64(x), pu.bf16_tensor_to_f64(w), *m.tab,
                                                pos.cpu().numpy(), 1e-6, False, pu.bf16_tensor_to_f64(g))
        # half a bf16 step of the value, and fp32 roundings of terms no larger
        # than a few times the largest value (2^-15 of it)
        assert np.all(np.abs(pu.bf16_tensor_to_f64(dx) - rx) <= 2.0 ** -8 * np.abs(rx) + 2.0 ** -15 * np.max(np.abs(rx)))
        # 2^-17 of the terms' magnitudes, which the rotation can raise by up to sqrt(2)
        assert np.all(np.abs(dwx.cpu().numpy() - rw) <= 2.0 ** -16 * np.max(mag))


def steps():
    """One call of each entry point with waits, on small inputs, with all buffers made beforehand."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    lens = [300, 1, 150]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    T = sum(lens)
    q, k, v, do = rnd(T, H, D), rnd(T, HK, D), rnd(T, HK, D), rnd(T, H, D)
    o, lse = torch.empty_like(q), torch.empty(H, T, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(binding.fa_bwd_workspace_size(3, H, 300, D), dtype=torch.uint8, device="cuda")
    args = (cu, cu, 300, 300, 0.1, True)
    big = torch.arange(0, 41, dtype=torch.int32, device="cuda") * 100  # more key blocks than SMs: no clusters
    qb, kb, vb = rnd(4000, 8, D), rnd(4000, 8, D), rnd(4000, 8, D)
    ob, lb = torch.empty_like(qb), torch.empty(8, 4000, device="cuda")
    gb = [torch.empty_like(qb) for _ in range(3)]
    wb = torch.empty(binding.fa_bwd_workspace_size(40, 8, 100, D), dtype=torch.uint8, device="cuda")
    out = {
        "forward": lambda: binding.fa_fwd_varlen_gqa(q, k, v, o, lse, *args),
        "backward": lambda: binding.fa_bwd_varlen_gqa(q, k, v, o, lse, do, dq, dk, dv, *args, ws),
        "backward det": lambda: binding.fa_bwd_varlen_gqa_deterministic(q, k, v, o, lse, do, dq, dk, dv, *args, ws),
        "forward big": lambda: binding.fa_fwd_varlen_gqa(qb, kb, vb, ob, lb, big, big, 100, 100, 0.1, True),
        "backward big": lambda: binding.fa_bwd_varlen_gqa(qb, kb, vb, ob, lb, qb, *gb, big, big, 100, 100, 0.1, True, wb),
    }
    for name, n in (("few", 3), ("many", 40)):  # streamed, and in tensor-core tiles
        dec = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in
               ([[0, 1, 2, 3]], [250], [0, n], [[4 + i] for i in range(n)], [1 + i % 60 for i in range(n)])]
        kp, vp, qd = rnd(4 + n, PAGE, HK, D), rnd(4 + n, PAGE, HK, D), rnd(n, H, D)
        od, ld = torch.empty_like(qd), torch.empty(n, H, device="cuda")
        wd = torch.empty(binding.fa_decode_shared_prefix_workspace_size(1, n, H, HK, D, n, 250, 60), dtype=torch.uint8,
                         device="cuda")
        out["decode " + name] = lambda a=(qd, kp, vp, od, ld, *dec, n, 250, 60, 0.1, wd): binding.fa_decode_shared_prefix(*a)
    return out


def test_waits_run_out_then_context_recovers(monkeypatch):
    """Dropped loads with a 2 ms bound (see the tests of the other kernels'
    waits): every kernel gives up, says so, and the context computes again."""
    import torch
    todo = steps()
    for f in todo.values():
        f()
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    monkeypatch.setenv("FA_TEST_WAIT_LIMIT_NS", "2000000")
    monkeypatch.setenv("FA_TEST_DROP_LOADS", "1")
    for name, f in todo.items():
        f()
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_ERR_TIMEOUT, name
    monkeypatch.delenv("FA_TEST_WAIT_LIMIT_NS")
    monkeypatch.delenv("FA_TEST_DROP_LOADS")
    for name, f in todo.items():
        f()
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK, name
    test_prompts_then_shared_decoding()


def test_entry_points_allocate_nothing():
    import torch
    todo = steps()
    m = Model(8300)
    q, k, v, pos = m.project(np.arange(50))
    yq, yk = torch.empty(50, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(50, HK, D, dtype=torch.bfloat16, device="cuda")
    gq, gk, dw = torch.empty_like(yq), torch.empty_like(yk), [torch.empty(D, device="cuda") for _ in range(2)]
    ws = torch.empty(binding.fa_qk_norm_rope_bwd_workspace_size(50, H, HK, D), dtype=torch.uint8, device="cuda")
    rope = (q, k, *m.w, m.cos, m.sin, pos)
    todo["rope"] = lambda: binding.fa_qk_norm_rope(*rope, yq, yk)
    todo["rope backward"] = lambda: binding.fa_qk_norm_rope_bwd(*rope, yq, yk, gq, gk, *dw, workspace=ws)
    for f in todo.values():  # first calls load modules and set kernel attributes
        f()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    for _ in range(5):
        for f in todo.values():
            f()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == before
