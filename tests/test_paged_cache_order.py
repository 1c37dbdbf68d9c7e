"""The paged cache's operators behind whatever stands in front of them on their
stream: copies, fills, another stream's work, nothing; eager and captured. Their
kernels are launched programmatically, so each must wait for all of it."""
import pytest

from exact_io_aware_29_gb300 import binding, build
import test_decode_q4 as dq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


T, H, HK, D, PAGE, BLOCKS = 3000, 8, 2, 128, 64, 60


class Chain:
    """append -> gather -> decode with inputs that change right in front of them."""

    def __init__(self):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(11)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
        self.src = [rnd(T, H + 2 * HK, D) for _ in range(2)]
        self.qkv = torch.zeros_like(self.src[0])
        self.slots_src = torch.randperm(BLOCKS * PAGE, device="cuda", generator=g)[:T].to(torch.int32)
        self.slots = torch.full_like(self.slots_src, -1)
        self.cache = binding.kv_cache_q4(BLOCKS, HK, PAGE, D)
        self.table = torch.arange(BLOCKS, dtype=torch.int32, device="cuda").view(1, -1)
        self.cu = torch.tensor([0, BLOCKS * PAGE], dtype=torch.int32, device="cuda")
        self.lens, self.want_lens = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        self.want_lens += BLOCKS * PAGE
        self.q_out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
        self.k, self.v = (torch.empty(BLOCKS * PAGE, HK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q1, self.o, self.lse = rnd(1, H, D), torch.empty(1, H, D, dtype=torch.bfloat16, device="cuda"), \
            torch.empty(1, H, device="cuda")
        self.ws = torch.empty(binding.fa_decode_paged_q4_workspace_size(1, 1, H, HK, D, BLOCKS * PAGE), dtype=torch.uint8,
                              device="cuda")
        self.big = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
        self.i = 0

    def outputs(self):
        return self.q_out, self.k, self.v, self.o, self.lse, *self.cache

    def run(self, other=None):
        """other: a stream that brings some of the inputs, joined by an event."""
        import torch
        here = torch.cuda.current_stream()
        for t in self.cache:
            t.zero_()
        if other is None:
            self.big.zero_()
            self.slots.copy_(self.slots_src)
            self.qkv.copy_(self.src[self.i])
        else:
            other.wait_stream(here)
            with torch.cuda.stream(other):
                self.big.zero_()
                self.qkv.copy_(self.src[self.i])
            self.slots.copy_(self.slots_src)
            here.wait_stream(other)
        binding.fa_kv_append_q4(self.qkv[:, :H], self.qkv[:, H:H + HK], self.qkv[:, H + HK:], None, None, None,
                                self.slots, self.q_out, *self.cache)
        binding.fa_kv_gather_q4(*self.cache, self.table, None, self.cu, self.k, self.v)
        self.lens.copy_(self.want_lens)
        binding.fa_decode_paged_q4(self.q1, *self.cache, self.o, self.lse, self.table, self.lens, BLOCKS * PAGE, D ** -0.5,
                                   self.ws)
        # The next call's work over this one's inputs and outputs, right behind it.
        keep = [t.clone() for t in self.outputs()]
        self.qkv.fill_(float("nan"))
        self.slots.fill_(-1)
        self.lens.zero_()
        return keep

    def expect(self):
        """Of the last inputs, with a wait for everything between the steps."""
        import torch
        x, sync = self.src[self.i], torch.cuda.synchronize
        cache = binding.kv_cache_q4(BLOCKS, HK, PAGE, D)
        sync()
        q = binding.kv_append_q4(x[:, :H], x[:, H:H + HK], x[:, H + HK:], None, None, None, self.slots_src, *cache)
        sync()
        k, v = binding.kv_gather_q4(*cache, self.table, None, self.cu, BLOCKS * PAGE)
        sync()
        o, lse = binding.attention_decode_paged_q4(self.q1, *cache, self.table, self.want_lens, BLOCKS * PAGE, D ** -0.5)
        sync()
        assert torch.equal(q, x[:, :H])
        return q, k, v, o, lse, *cache


@pytest.mark.parametrize("streams", [1, 2])
def test_eager(streams):
    import torch
    c = Chain()
    other = torch.cuda.Stream() if streams == 2 else None
    for i in (0, 1, 0, 1):
        c.i = i
        got = c.run(other)
        assert all(torch.equal(a, b) for a, b in zip(got, c.expect()))


@pytest.mark.parametrize("streams", [1, 2])
def test_captured(streams):
    import torch
    c = Chain()
    other = torch.cuda.Stream() if streams == 2 else None
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.run(other)
    torch.cuda.synchronize()
    graphs = []
    for i in (0, 1):
        c.i = i
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            keep = c.run(other)
        graphs.append((g, keep, i))
    for g, keep, i in graphs * 2:
        g.replay()
        torch.cuda.synchronize()
        c.i = i
        assert all(torch.equal(a, b) for a, b in zip(keep, c.expect()))


def test_first_in_a_graph():
    """Each operator as the only node of a graph, replayed back to back."""
    import torch
    c = Chain()
    c.qkv.copy_(c.src[0])
    c.slots.copy_(c.slots_src)
    c.lens.copy_(c.want_lens)
    calls = [
        lambda: binding.fa_kv_append_q4(c.qkv[:, :H], c.qkv[:, H:H + HK], c.qkv[:, H + HK:], None, None, None, c.slots,
                                        c.q_out, *c.cache),
        lambda: binding.fa_kv_gather_q4(*c.cache, c.table, None, c.cu, c.k, c.v),
        lambda: binding.fa_decode_paged_q4(c.q1, *c.cache, c.o, c.lse, c.table, c.lens, BLOCKS * PAGE, D ** -0.5, c.ws)]
    graphs = []
    for f in calls:
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for _ in range(3):
        for t in c.outputs():
            t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        c.i = 0
        assert all(torch.equal(a, b) for a, b in zip(c.outputs(), c.expect()))


def test_two_graphs_that_share_a_workspace_one_after_the_other():
    """Steps of different shapes whose parts lie in the same workspace, replayed
    in turn on one stream: no call's parts are overwritten before they are joined."""
    import torch
    xs = [dq.Step(lens, n, 8, 2, 128, 64, 8900 + n, bound=40000) for lens, n in (([9000, 4000], 1), ([7000, 100, 2], 2))]
    want = [x.run() for x in xs]
    ws = torch.empty(max(binding.fa_decode_paged_q4_workspace_size(x.B, x.n, 8, 2, 128, 40000) for x in xs),
                     dtype=torch.uint8, device="cuda")
    out = [(torch.empty_like(x.q), torch.empty(*x.q.shape[:-1], device="cuda")) for x in xs]
    args = [x.args() for x in xs]
    torch.cuda.synchronize()
    graphs = []
    for a, (o, lse) in zip(args, out):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                binding.fa_decode_paged_q4(*a[:5], o, lse, *a[5:], ws)
        graphs.append(g)
    for _ in range(5):
        for o, lse in out:
            o.zero_(), lse.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (o, lse), (wo, wl) in zip(out, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
    for x, w in zip(xs, want):
        x.check(*w)
