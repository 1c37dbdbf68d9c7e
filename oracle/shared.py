"""fp64 oracle of the shared-prefix decoding step (test infrastructure only)."""
from __future__ import annotations

import numpy as np

from .attention import NEG_INF, gather_pages


def shared_prefix_decode_forward(q, k_pool, v_pool, prefix_table, prefix_lens, cu_seqs, block_table, seq_lens, scale):
    """q [B, H, d]; pools [num_blocks, block_size, H_kv, d]. Returns O [B, H, d],
    LSE [B, H] and A [B, H, d] = sum of P |V| (what rounding errors of O scale
    with): per sequence, the keys of its prefix and its own, concatenated."""
    q = np.asarray(q, np.float64)
    B, H, d = q.shape
    bs, Hk = np.asarray(k_pool).shape[1:3]
    o, a, lse = np.zeros((B, H, d)), np.zeros((B, H, d)), np.full((B, H), NEG_INF)
    owner = {b: p for p in range(len(cu_seqs) - 1) for b in range(int(cu_seqs[p]), int(cu_seqs[p + 1]))}
    for b in range(B):
        parts = [(block_table[b], int(seq_lens[b]))]
        if b in owner:
            parts.insert(0, (prefix_table[owner[b]], int(prefix_lens[owner[b]])))
        k, v = (np.concatenate([np.asarray(gather_pages(pool, t, n, bs), np.float64).reshape(n, Hk, d)
                                for t, n in parts]) for pool in (k_pool, v_pool))
        if not len(k):
            continue
        for h in range(H):
            x = scale * (k[:, h * Hk // H] @ q[b, h])
            m = np.max(x)
            p = np.exp(x - m)
            z = np.sum(p)
            o[b, h], a[b, h], lse[b, h] = p @ v[:, h * Hk // H] / z, p @ np.abs(v[:, h * Hk // H]) / z, m + np.log(z)
    return o, lse, a
