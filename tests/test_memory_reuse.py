"""Memory that changes hands between two calls on one stream. A forward's
inputs or outputs may be dropped as soon as the call has returned, and a
caching allocator hands their memory straight to the next call on the stream,
say as a backward's workspace. The backward's first kernel is launched while
the forward still runs; it must leave the workspace alone until then. Here the
workspace lies over the key, value or output tensors of the forward in front
of it, for every pair of layouts. Each result must equal, bit for bit, that of
the same calls with nothing in flight (the deterministic order; dK and dV of
the default one)."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def _normal(seed, *shapes):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16) for s in shapes]


class Problem:
    """One problem of a layout: its tensors and the calls on them."""

    def __init__(self, layout, seed, B, H, N, d):
        import torch
        self.layout, self.scale = layout, d ** -0.5
        Hk = H // 4 if layout == "grouped" else H
        qs, ks = ((B, H, N, d),) * 2 if layout == "fixed" else ((B * N, H, d), (B * N, Hk, d))
        self.q, self.k, self.v, self.do = _normal(seed, qs, ks, ks, qs)
        self.o = torch.empty_like(self.q)
        self.lse = torch.empty((B, H, N) if layout == "fixed" else (H, B * N), device="cuda")
        cu = torch.from_numpy(np.arange(B + 1, dtype=np.int32) * N).cuda()
        self.rest = (self.scale, True) if layout == "fixed" else (cu, cu, N, N, self.scale, True)
        self.ws_bytes = binding.fa_bwd_workspace_size(B, H, N, d)

    def forward(self):
        fn = {"fixed": binding.fa_fwd, "packed": binding.fa_fwd_varlen, "grouped": binding.fa_fwd_varlen_gqa}
        fn[self.layout](self.q, self.k, self.v, self.o, self.lse, *self.rest)

    def backward(self, ws, deterministic):
        import torch
        name = {"fixed": "fa_bwd", "packed": "fa_bwd_varlen", "grouped": "fa_bwd_varlen_gqa"}[self.layout]
        fn = getattr(binding, name + ("_deterministic" if deterministic else ""))
        grads = [torch.empty_like(t) for t in (self.q, self.k, self.v)]
        fn(self.q, self.k, self.v, self.o, self.lse, self.do, *grads, *self.rest, workspace=ws)
        return grads


LAYOUTS = ["fixed", "packed", "grouped"]


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("bwd", LAYOUTS)
@pytest.mark.parametrize("fwd", LAYOUTS)
def test_workspace_over_the_tensors_of_the_forward_in_front(fwd, bwd, deterministic):
    import torch
    a, b = Problem(fwd, 1, 2, 16, 3000, 128), Problem(bwd, 2, 4, 16, 1024, 128)
    b.forward()
    want_grads = b.backward(torch.empty(b.ws_bytes, dtype=torch.uint8, device="cuda"), deterministic)
    a.forward()
    torch.cuda.synchronize()
    want_o, want_lse, kept = a.o.clone(), a.lse.clone(), {n: getattr(a, n).clone() for n in "kvo"}
    buf = torch.empty(max(b.ws_bytes, sum(t.numel() * 2 + 256 for t in kept.values())), dtype=torch.uint8, device="cuda")
    for moved in ("kv", "o", "kvo"):
        at = 0
        for n, t in kept.items():
            if n in moved:
                view = buf[at:at + t.numel() * 2].view(torch.bfloat16).view(t.shape)
                at += -(-t.numel() * 2 // 256) * 256
            else:
                view = torch.empty_like(t)
            setattr(a, n, view)
        for _ in range(3):
            for n, t in kept.items():
                getattr(a, n).copy_(t)
            torch.cuda.synchronize()
            a.forward()
            grads = b.backward(buf[:b.ws_bytes], deterministic)
            torch.cuda.synchronize()
            assert binding.fa_check_status() == binding.FA_OK
            assert torch.equal(a.lse, want_lse)
            if "o" not in moved:
                assert torch.equal(a.o, want_o)
            for g, w in list(zip(grads, want_grads))[0 if deterministic else 1:]:
                assert torch.equal(g, w)
            # dQ of the default order: sums of the same fp32 terms in another
            # order, rounded once more: two bf16 steps of the largest.
            top = float(want_grads[0].float().abs().max())
            assert float((grads[0].float() - want_grads[0].float()).abs().max()) <= 2.0 ** -7 * top
