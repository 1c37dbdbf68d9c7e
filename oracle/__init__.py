"""CPU oracle for exact attention (fp64).

TEST INFRASTRUCTURE ONLY: imported by the tests, by the smoke check and by the
benchmark's CPU-baseline leg, never by the product path. Nothing here calls or
imports the CUDA library, and the CUDA library shares no code with it.
"""
from .attention import (  # noqa: F401
    attention_backward,
    attention_backward_rows,
    attention_forward,
    attention_forward_rows,
    batched_backward,
    batched_forward,
    blocked_attention_forward,
    gather_pages,
    merge_states,
    online_softmax_state,
    paged_decode_forward,
    probabilities,
    safe_softmax,
    softmax_grad,
    varlen_backward,
    varlen_forward,
    visible,
)
from .norm_rope import norm_rope_backward, norm_rope_forward  # noqa: F401
from .shared import shared_prefix_decode_forward  # noqa: F401
from .kv_cache import (  # noqa: F401
    held_q4,
    held_q4_bf16,
    q4_decode_forward,
    quantise_q4,
    rotated,
    to_bf16,
    unpack_codes,
)
