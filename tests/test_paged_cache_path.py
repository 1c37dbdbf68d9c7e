"""The paged cache's operators as a server uses them, one after the other:
prompts -> rotation and append -> prompt attention; the same prompts continued
behind the cache; generated tokens -> append -> decoding steps, drafts among
them. In 4 bits, and beside it in bf16 with the decoders that were there. Each
attention is compared with the fp64 oracle on what the cache holds, with the
tolerances of its own tests."""
import numpy as np
import pytest

import oracle
from exact_io_aware_29_gb300 import binding, build
import parity_util as pu

pytestmark = pytest.mark.gpu
H, HK, D, PAGE, POOL = 8, 2, 128, 64, 40


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


class Server:
    """Sequences with pages of their own in both caches, and fp64 copies of
    what each cache stands for, slot by slot."""

    def __init__(self, B, width, seed):
        import torch
        self.rng = np.random.default_rng(seed)
        self.table = self.rng.permutation(POOL)[:B * width].reshape(B, width).astype(np.int32)
        self.dev_table = torch.from_numpy(self.table).cuda()
        self.lens = np.zeros(B, np.int64)
        angle = np.arange(600)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
        self.tab = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        self.cos, self.sin = (torch.from_numpy(t).cuda() for t in self.tab)
        nan = lambda: torch.full((POOL, PAGE, HK, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.bf16, self.q4 = [nan(), nan()], binding.kv_cache_q4(POOL, HK, PAGE, D)
        for t in self.q4[1::2]:
            t.fill_(float("nan"))
        self.held = {"bf16": [np.full((POOL * PAGE, HK, D), np.nan) for _ in range(2)],
                     "q4": [np.full((POOL * PAGE, HK, D), np.nan) for _ in range(2)]}
        self.scale = D ** -0.5

    def slots(self, b, first, count):
        t = first + np.arange(count)
        return self.table[b, t // PAGE].astype(np.int64) * PAGE + t % PAGE

    def append(self, new):
        """new[b] tokens of each sequence through both caches: the rotated queries."""
        import torch
        T = int(np.sum(new))
        qkv = torch.from_numpy(self.rng.standard_normal((T + 2, H + 2 * HK, D)).astype(np.float32)).to(torch.bfloat16).cuda()
        pos = np.concatenate([self.lens[b] + np.arange(n) for b, n in enumerate(new)] + [[0, 0]]).astype(np.int32)
        slots = np.concatenate([self.slots(b, self.lens[b], n) for b, n in enumerate(new)] + [[-1, -1]]).astype(np.int32)
        args = (qkv[:, :H], qkv[:, H:H + HK], qkv[:, H + HK:], self.cos, self.sin,
                *(torch.from_numpy(x).cuda() for x in (pos, slots)))
        q = binding.kv_append(*args, *self.bf16)
        assert torch.equal(q, binding.kv_append_q4(*args, *self.q4))
        f = pu.bf16_tensor_to_f64(qkv)
        rq, rk = (oracle.rotated(x, *self.tab, pos, False)[:T] for x in (f[:, :H], f[:, H:H + HK]))
        assert np.array_equal(pu.bf16_tensor_to_f64(q)[:T], rq)
        for i, rows in enumerate((rk, f[:T, H + HK:])):
            self.held["bf16"][i][slots[:T]] = rows
            self.held["q4"][i][slots[:T]] = oracle.held_q4(*oracle.quantise_q4(rows))
        self.lens = self.lens + np.asarray(new)
        return q[:T]

    def values(self, kind, b):
        at = self.slots(b, 0, int(self.lens[b]))
        return [x[at] for x in self.held[kind]]

    def i32(self, x):
        import torch
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def prompt(self, q, new):
        """Attention of the newest tokens over all of the 4-bit cache's, read back."""
        cq, ck = (np.concatenate([[0], np.cumsum(n)]) for n in (new, self.lens))
        k, v = binding.kv_gather_q4(*self.q4, self.dev_table, None, self.i32(ck), int(ck[-1]))
        for i, x in enumerate((k, v)):
            want = np.concatenate([self.values("q4", b)[i] for b in range(len(new))])
            assert np.array_equal(pu.bf16_tensor_to_f64(x), oracle.to_bf16(want))
        o, lse = binding.attention_forward_varlen_gqa(q, k, v, self.i32(cq), self.i32(ck), max(new), int(max(self.lens)),
                                                      self.scale, True)
        rep = lambda x: np.repeat(pu.bf16_tensor_to_f64(x), H // HK, axis=1)  # noqa: E731
        ro, rl = oracle.varlen_forward(pu.bf16_tensor_to_f64(q), rep(k), rep(v), cq, ck, self.scale, True)
        assert pu.o_err(pu.bf16_tensor_to_f64(o), ro) <= pu.O_ATOL
        assert pu.max_abs(lse.cpu().numpy(), rl) <= pu.LSE_ATOL

    def decode(self, q, n):
        """n new queries of each sequence over each cache."""
        import torch
        B = len(self.lens)
        q, most = q.view(B, n, H, D), int(max(self.lens))
        got = {"q4": binding.attention_decode_paged_q4(q, *self.q4, self.dev_table, self.i32(self.lens), most, self.scale)}
        if n == 1:
            none = (self.i32([[0]]), self.i32([0]), self.i32([0, 0]))
            o, lse = binding.attention_decode_shared_prefix(q[:, 0].contiguous(), *self.bf16, *none, self.dev_table,
                                                            self.i32(self.lens), 1, 1, most, self.scale)
            got["bf16"] = o[:, None], lse[:, None]
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        for kind, (o, lse) in got.items():
            k, v = ([self.values(kind, b)[i] for b in range(B)] for i in range(2))
            ro, rl, _ = oracle.q4_decode_forward(pu.bf16_tensor_to_f64(q), k, v, self.lens, self.scale)
            assert pu.o_err(pu.bf16_tensor_to_f64(o), ro) <= pu.O_ATOL
            assert pu.max_abs(lse.cpu().numpy(), rl) <= pu.LSE_ATOL


def test_prompts_continuations_and_generation():
    s = Server(3, 6, 61)
    new = [130, 64, 1]
    s.prompt(s.append(new), new)          # the prompts
    for _ in range(3):
        s.decode(s.append([1, 1, 1]), 1)  # tokens generated one by one
    new = [40, 1, 99]
    s.prompt(s.append(new), new)          # another turn behind the cache
    s.decode(s.append([5, 5, 5]), 5)      # drafts looked over at once
    s.lens = s.lens - [3, 0, 5]           # some of them not taken
    s.decode(s.append([1, 1, 1]), 1)
