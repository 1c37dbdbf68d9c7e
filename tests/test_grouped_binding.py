"""What the Python binding of the grouped-head operators refuses before it
calls the library: tensors not on a GPU, of another dtype or shape, strided
where they must not be, and streams of another device."""
import numpy as np
import pytest

from exact_io_aware_29_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load_library()


def calls(device):
    """Entry point -> (function, its tensors by name, the rest by name)."""
    import torch
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    q, k = t(9, 4, 64), t(9, 2, 64)
    packed = dict(q=q, k=k, v=t(9, 2, 64), o=t(9, 4, 64), lse=t(4, 9, dt=torch.float32))
    cu = dict(cu_seqlens_q=i(0, 4, 9), cu_seqlens_k=i(0, 4, 9))
    sizes = dict(max_seqlen_q=5, max_seqlen_k=5, scale=0.1, causal=True)
    grads = dict(dO=t(9, 4, 64), dq=t(9, 4, 64), dk=t(9, 2, 64), dv=t(9, 2, 64))
    rope = dict(q=q, k=k, q_weight=t(64), k_weight=t(64), cos=t(16, 32, dt=torch.float32),
                sin=t(16, 32, dt=torch.float32), positions=torch.arange(9, dtype=torch.int32, device=device))
    cache = t(4, 64, 2, 64)
    return {
        "fa_fwd_varlen_gqa": (binding.fa_fwd_varlen_gqa, {**packed, **cu}, sizes),
        "fa_bwd_varlen_gqa": (binding.fa_bwd_varlen_gqa, {**packed, **grads, **cu}, sizes),
        "fa_bwd_varlen_gqa_deterministic": (binding.fa_bwd_varlen_gqa_deterministic, {**packed, **grads, **cu}, sizes),
        "fa_qk_norm_rope": (binding.fa_qk_norm_rope, {**rope, "q_out": t(9, 4, 64), "k_out": t(9, 2, 64)}, {}),
        "fa_qk_norm_rope_bwd": (binding.fa_qk_norm_rope_bwd, {
            **rope, "dq_out": t(9, 4, 64), "dk_out": t(9, 2, 64), "dq": t(9, 4, 64), "dk": t(9, 2, 64),
            "dq_weight": t(64, dt=torch.float32), "dk_weight": t(64, dt=torch.float32)}, {}),
        "fa_decode_shared_prefix": (binding.fa_decode_shared_prefix, dict(
            q=q, k_cache=cache, v_cache=cache.clone(), o=t(9, 4, 64), lse=t(9, 4, dt=torch.float32),
            prefix_table=i(0, 1).view(1, 2), prefix_lens=i(100), cu_prefix_seqs=i(0, 9),
            block_table=i(*([2] * 9)).view(9, 1), seq_lens=i(*range(9))),
            dict(max_group=9, max_prefix_len=128, max_seq_len=64, scale=0.1)),
    }


NAMES = ["fa_fwd_varlen_gqa", "fa_bwd_varlen_gqa", "fa_bwd_varlen_gqa_deterministic", "fa_qk_norm_rope",
         "fa_qk_norm_rope_bwd", "fa_decode_shared_prefix"]


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
    strided = {"fa_qk_norm_rope": ("q", "k"), "fa_qk_norm_rope_bwd": ("q", "k", "dq", "dk")}.get(name, ())
    for arg, t in tensors.items():
        for what, bad in (
                ("host", t.cpu()),
                ("dtype", t.to(torch.float16 if t.is_floating_point() else torch.int64)),
                ("shape", torch.cat((t, t))[:-1] if t.shape[0] > 1 else torch.cat((t, t))),
                ("rank", t[None]),
                ("strided", torch.stack((t, t), -1)[..., 0])):
            if what == "shape" and arg in ("cos", "cu_seqlens_q", "k_cache", "prefix_table") and bad.shape[1:] == t.shape[1:]:
                continue  # this tensor's length is what the others are held against, or is its own
            if what == "strided" and bad.is_contiguous():
                continue  # one element
            if what == "strided" and arg in strided:
                bad = torch.stack((t, t), 1)[:, 0].transpose(1, 2)  # heads not side by side
            with pytest.raises((ValueError, IndexError)):
                fn(**{**tensors, arg: bad}, **rest)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK


@pytest.mark.gpu
def test_workspaces_on_the_host_are_refused():
    import torch
    for name in ("fa_bwd_varlen_gqa", "fa_qk_norm_rope_bwd", "fa_decode_shared_prefix"):
        fn, tensors, rest = calls("cuda")[name]
        with pytest.raises(ValueError, match="workspace"):
            fn(**tensors, **rest, workspace=torch.empty(1 << 24, dtype=torch.uint8))
        with pytest.raises(binding.FaError):
            fn(**tensors, **rest, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
def test_outputs_belong_to_the_stream_of_the_call():
    """A call on another stream than the current one allocates there: while the
    current stream still works on a tensor that has died, its memory is not
    handed to the call."""
    import torch
    fn, x, rest = calls("cuda")["fa_qk_norm_rope"]
    s = torch.cuda.Stream()
    args = [x[n] for n in ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions")]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        a = torch.empty_like(x["q"])
    ptr = a.data_ptr()
    del a
    y, _ = binding.qk_norm_rope(*args, stream=s)
    assert y.data_ptr() == ptr  # from the stream's own pool
    torch.cuda.synchronize()
