"""Check mode (FA_CHECK=1, read once per process, hence a child process): the
grouped-head entry points refuse offsets, lengths, tables and positions that
break their contracts on the host, before anything runs, and accept good ones."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
from exact_io_aware_29_gb300 import binding as fa

def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")

def rnd(*s):
    return torch.randn(*s, device="cuda").to(torch.bfloat16)

def refused(f):
    try:
        f()
    except fa.FaError as e:
        assert e.status == fa.FA_ERR_INVALID, e
        return
    raise AssertionError("accepted")

q, k, v = rnd(100, 4, 64), rnd(100, 2, 64), rnd(100, 2, 64)
def packed(cq, ck, mq=60, mk=60):
    o, lse = fa.attention_forward_varlen_gqa(q, k, v, cq, ck, mq, mk, 0.1, True)
    fa.attention_backward_varlen_gqa(q, k, v, o, lse, q, cq, ck, mq, mk, 0.1, True)
good = i32(0, 60, 100)
packed(good, good)
packed(i32(0, 60, 90), good)                          # rows of no sequence at the end
refused(lambda: packed(i32(0, 60, 101), good))       # ends past total_q
refused(lambda: packed(good, i32(5, 60, 100)))       # does not start at 0
refused(lambda: packed(i32(0, 61, 100), good))       # longer than max_seqlen_q
refused(lambda: packed(good, i32(0, 70, 60, 100)[:3].clone()))

t = torch.ones(10, 16, device="cuda")
w = rnd(64)
def rope(pos):
    fa.qk_norm_rope(q, k, w, w, t, t, pos)
    fa.qk_norm_rope_backward(q, k, w, w, t, t, pos, q, k)
pos = torch.arange(100, dtype=torch.int32, device="cuda") % 10
rope(pos)
refused(lambda: rope(pos + 1))
refused(lambda: rope(pos - 1))

cache = rnd(6, 64, 2, 64)
qd = rnd(3, 4, 64)
def decode(ptab=i32(0, 1).view(1, 2), plens=i32(100), cu=i32(0, 3), tab=i32(2, 3, 4).view(3, 1), lens=i32(64, 0, 5)):
    fa.attention_decode_shared_prefix(qd, cache, cache, ptab, plens, cu, tab, lens, 3, 128, 64, 0.1)
decode()
decode(cu=i32(1, 2))                                  # sequences of no prefix
decode(tab=i32(2, 99, 4).view(3, 1))                  # an entry that is not read
refused(lambda: decode(ptab=i32(0, 6).view(1, 2)))
refused(lambda: decode(plens=i32(129)))
refused(lambda: decode(cu=i32(0, 4)))
refused(lambda: decode(cu=i32(2, 1)))
refused(lambda: decode(tab=i32(-1, 3, 4).view(3, 1)))
refused(lambda: decode(lens=i32(65, 0, 5)))
print("done")
"""


def test_contracts_are_checked_on_the_host():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env={**os.environ, "FA_CHECK": "1"}, text=True,
                       capture_output=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]
