"""What the Python binding of the paged cache's operators refuses before it
calls the library (tensors not on a GPU, of another dtype or shape, strided
where they must not be; see test_grouped_binding.py), and check mode: contracts
of device data that the host verifies (FA_CHECK=1, read once per process)."""
import os
import subprocess
import sys

import pytest

from exact_io_aware_29_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def calls(device):
    """Entry point -> (function, its tensors by name, the rest by name)."""
    import torch
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    new = dict(q=t(9, 4, 128), k=t(9, 2, 128), v=t(9, 2, 128), cos=t(16, 32, dt=torch.float32),
               sin=t(16, 32, dt=torch.float32), positions=i(*range(9)), slots=i(*range(9)), q_out=t(9, 4, 128))
    codes, scales = t(3, 2, 16, 64, dt=torch.uint8), t(3, 2, 16, 2, 2)
    q4 = dict(k_codes=codes, k_scales=scales, v_codes=codes.clone(), v_scales=scales.clone())
    return {
        "fa_kv_append": (binding.fa_kv_append, {**new, "k_cache": t(3, 16, 2, 128), "v_cache": t(3, 16, 2, 128)}, {}),
        "fa_kv_append_q4": (binding.fa_kv_append_q4, {**new, **q4}, {}),
        "fa_kv_gather_q4": (binding.fa_kv_gather_q4, dict(
            **q4, block_table=i(0, 1, 2, 0).view(2, 2), starts=i(0, 3), cu_seqlens_k=i(0, 4, 9), k=t(9, 2, 128),
            v=t(9, 2, 128)), {}),
        "fa_decode_paged_q4": (binding.fa_decode_paged_q4, dict(
            **{**q4, "q": t(2, 3, 4, 128)}, o=t(2, 3, 4, 128), lse=t(2, 3, 4, dt=torch.float32),
            block_table=i(0, 1, 2, 0).view(2, 2), seq_lens=i(30, 5)), dict(max_seq_len=32, scale=0.1)),
    }


NAMES = ["fa_kv_append", "fa_kv_append_q4", "fa_kv_gather_q4", "fa_decode_paged_q4"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_the_host_are_refused(name):
    fn, tensors, rest = calls("cpu")[name]
    with pytest.raises(ValueError, match="CUDA"):
        fn(**tensors, **rest)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_checked(name):
    import torch
    fn, tensors, rest = calls("cuda")[name]
    fn(**tensors, **rest)  # as they are, they are accepted
    torch.cuda.synchronize()
    for arg, t in tensors.items():
        other = torch.float16 if t.is_floating_point() else (torch.int8 if t.dtype == torch.uint8 else torch.int64)
        for what, bad in (
                ("host", t.cpu()),
                ("dtype", t.to(other)),
                ("shape", torch.cat((t, t))[:-1]),
                ("last", torch.cat((t, t), -1)),
                ("rank", t[None]),
                ("strided", torch.stack((t, t), -1)[..., 0])):
            if what == "shape" and arg in ("cos", "k", "k_cache", "k_codes", "block_table", "q"):
                continue  # this tensor's length is what the others are held against, or is its own
            if what == "last" and arg == "block_table":
                continue  # so is a table's width
            with pytest.raises((ValueError, IndexError)):
                fn(**{**tensors, arg: bad}, **rest)
    # Heads that do not lie side by side.
    for arg in ("q", "k", "v"):
        if name.startswith("fa_kv_append"):
            with pytest.raises(ValueError):
                fn(**{**tensors, arg: torch.stack((tensors[arg],) * 2, 1)[:, 0].transpose(1, 2)})
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK


@pytest.mark.gpu
def test_optional_tensors_go_together():
    for name in ("fa_kv_append", "fa_kv_append_q4"):
        fn, x, _ = calls("cuda")[name]
        for gone in (("q",), ("q_out",), ("cos",), ("sin",), ("positions",)):
            with pytest.raises(ValueError):
                fn(**{**x, **dict.fromkeys(gone)})
        for gone in (("q", "q_out"), ("cos", "sin"), ("cos", "sin", "positions")):
            fn(**{**x, **dict.fromkeys(gone)})


@pytest.mark.gpu
def test_workspaces_are_checked():
    import torch
    fn, x, rest = calls("cuda")["fa_decode_paged_q4"]
    with pytest.raises(ValueError, match="workspace"):
        fn(**x, **rest, workspace=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(binding.FaError):
        fn(**x, **rest, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


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

q, k, v = rnd(5, 4, 64), rnd(5, 2, 64), rnd(5, 2, 64)
t = torch.ones(10, 16, device="cuda")
bf16 = [torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
q4 = fa.kv_cache_q4(3, 2, 16, 64)
def append(pos=i32(0, 1, 2, 3, 9), slots=i32(47, 0, 5, 6, 7)):
    fa.kv_append(q, k, v, t, t, pos, slots, *bf16)
    fa.kv_append_q4(q, k, v, t, t, pos, slots, *q4)
append()
append(slots=i32(-1, -1, 3, -7, 4))                # padding, more than once
refused(lambda: append(slots=i32(48, 0, 5, 6, 7)))
refused(lambda: append(slots=i32(5, 0, 5, 6, 7)))  # a slot twice
refused(lambda: append(pos=i32(0, 1, 2, 3, 10)))
refused(lambda: append(pos=i32(0, -1, 2, 3, 4)))

def gather(table=i32(2, 0, 1, 99).view(2, 2), starts=i32(3, 0), cu=i32(0, 29, 45)):
    fa.kv_gather_q4(*q4, table, starts, cu, 50)
gather()                                            # the second row's second page is not read
gather(starts=None)
gather(table=i32(-5, 0, 1, 99).view(2, 2), starts=i32(16, 0), cu=i32(0, 16, 20))
refused(lambda: gather(table=i32(3, 0, 1, 0).view(2, 2)))
refused(lambda: gather(starts=i32(4, 0)))           # past the row's pages
refused(lambda: gather(starts=i32(-1, 0)))
refused(lambda: gather(cu=i32(0, 30, 29)))
refused(lambda: gather(cu=i32(0, 20, 51)))

def decode(table=i32(2, 0, 1, 99).view(2, 2), lens=i32(32, 16)):
    fa.attention_decode_paged_q4(rnd(2, 3, 4, 64), *q4, table, lens, 32, 0.1)
decode()
decode(lens=i32(0, 1))
refused(lambda: decode(table=i32(2, -1, 1, 0).view(2, 2)))
refused(lambda: decode(lens=i32(33, 0)))
refused(lambda: decode(lens=i32(-1, 0)))
print("done")
"""


@pytest.mark.gpu
def test_contracts_are_checked_on_the_host():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env={**os.environ, "FA_CHECK": "1"}, text=True,
                       capture_output=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


EMPTY_CHILD = r"""
import torch
from exact_io_aware_29_gb300 import binding as fa

def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")

q4 = fa.kv_cache_q4(3, 2, 16, 64)
for starts in (5, 16, 32, 33, 2 ** 31 - 1, -1):
    # The first sequence has no rows: neither its start nor its pages are looked at.
    k, v = fa.kv_gather_q4(*q4, i32(-1, 99, 1, 0).view(2, 2), i32(starts, 3), i32(0, 0, 20), 20)
    assert not k.any() and not v.any()
try:
    fa.kv_gather_q4(*q4, i32(-1, 99, 1, 0).view(2, 2), i32(5, 3), i32(0, 1, 20), 20)
except fa.FaError as e:
    assert e.status == fa.FA_ERR_INVALID
    print("done")
"""


@pytest.mark.gpu
def test_a_gather_of_no_row_reads_no_page():
    r = subprocess.run([sys.executable, "-c", EMPTY_CHILD], cwd=ROOT, env={**os.environ, "FA_CHECK": "1"}, text=True,
                       capture_output=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("name", ["kv_append", "kv_append_q4"])
def test_without_queries_host_tensors_are_refused_like_others(name):
    x = {k: t for k, t in calls("cpu")["fa_" + name][1].items() if k != "q_out"}
    with pytest.raises(ValueError, match="CUDA"):
        getattr(binding, name)(**{**x, "q": None})


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["kv_append", "kv_append_q4"])
def test_the_forms_that_allocate_take_no_queries_too(name):
    import torch
    x = {k: t for k, t in calls("cuda")["fa_" + name][1].items() if k != "q_out"}
    caches = [k for k in x if k.startswith(("k_", "v_"))]
    for k in ("k", "v"):
        x[k].normal_()
    q = getattr(binding, name)(**x)
    want = [x[c].clone() for c in caches]
    assert q.shape == x["q"].shape and any(t.any() for t in want)
    for c in caches:
        x[c].zero_()
    assert getattr(binding, name)(**{**x, "q": None}) is None
    assert all(torch.equal(x[c], w) for c, w in zip(caches, want))


HUGE_CHILD = r"""
from exact_io_aware_29_gb300 import binding as fa

lib, x = fa.load_library(), 0x10000  # (nothing is read: the tables' copies come first, and there is no room for them)
for blocks in (1 << 30, 2 ** 31 - 1):  # tables of 2^50 entries and more
    st = [lib.fa_decode_paged_q4(*[x] * 9, 1 << 20, 1, 1, 1, 64, 10, 16, blocks, 64, 0.1, x, 1 << 60, None),
          lib.fa_decode_paged(*[x] * 7, 1 << 20, 1, 64, 10, 64, blocks, 64, 0.1, x, 1 << 60, None)]
    assert st == [fa.FA_ERR_UNSUPPORTED] * 2, st
print("done")
"""


def test_tables_that_the_host_has_no_room_for_are_refused():
    """Check mode copies them; no exception leaves a C entry."""
    r = subprocess.run([sys.executable, "-c", HUGE_CHILD], cwd=ROOT, env={**os.environ, "FA_CHECK": "1"}, text=True,
                       capture_output=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("name", [*NAMES, "kv_append", "kv_append_q4", "kv_cache_q4", "kv_gather_q4",
                                  "attention_decode_paged_q4", "fa_decode_paged_q4_workspace_size"])
def test_the_package_exports_them(name):
    import exact_io_aware_29_gb300 as package
    assert getattr(package, name) is getattr(binding, name)
