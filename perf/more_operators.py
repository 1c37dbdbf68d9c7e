"""What is measured of the operators that write and read a paged cache: tokens
appended with the position rotation on the way, to a cache of bf16 and to one
held in 4 bits, the 4-bit cache read back as packed keys and values, and
decoding steps over it.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, each output rounded once) or, with ``own`` set, through the
package's binding, as a user's program calls it. ``exact`` gives the same
outputs from the definitions in 64 bits.

The 4-bit cache: 64 consecutive elements of a key or value row share a scale s
and a minimum z (both bf16), and stand for z + s * code, code in 0..15, with
z = min, s = bf16((max - min) / 15) and code = (x - z) / s to the nearest
(ties to even). Two codes a byte, the even element's in the low half.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
NEG = float("-inf")
GROUP = 64


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One generated token for each of 64 sequences: latency.
        dict(name="append_step", op="append", tokens=64, batch=64, past=4000, pad=0, lens=1, heads=32, kv_heads=8,
             d=128, rot=128, interleaved=False, positions=32768, page=64),
        # A ragged batch with padding behind it, half of each head rotated, pairs side by side, small pages.
        dict(name="append_odd_d64", op="append", tokens=1001, batch=9, past=300, pad=23, lens=2, heads=12, kv_heads=4,
             d=64, rot=32, interleaved=True, positions=5000, page=16),
        # The prompts of a whole packed batch.
        dict(name="append_prompt", op="append", tokens=16384, batch=16, past=0, pad=0, lens=3, heads=32, kv_heads=8,
             d=128, rot=128, interleaved=False, positions=32768, page=64),
        # The same three for the 4-bit cache, what was written read back.
        dict(name="write_q4_step", op="write_q4", tokens=64, batch=64, past=4000, pad=0, lens=1, heads=32, kv_heads=8,
             d=128, rot=128, interleaved=False, positions=32768, page=64),
        dict(name="write_q4_odd_d64", op="write_q4", tokens=1001, batch=9, past=300, pad=23, lens=2, heads=12,
             kv_heads=4, d=64, rot=32, interleaved=True, positions=5000, page=16),
        dict(name="write_q4_prompt", op="write_q4", tokens=16384, batch=16, past=0, pad=0, lens=3, heads=32,
             kv_heads=8, d=128, rot=128, interleaved=False, positions=32768, page=64),
        # A few short sequences read back from somewhere inside, so that a prompt can be continued.
        dict(name="gather_short_d64", op="gather", batch=7, lo=1, hi=900, skip=100, lens=4, kv_heads=2, d=64, page=32),
        # The cached part of a packed batch of long prompts.
        dict(name="gather_long", op="gather", batch=16, lo=512, hi=8192, skip=0, lens=5, kv_heads=8, d=128, page=64),
        # One generated token for each of a few sequences that have just begun: latency.
        dict(name="decode_q4_few", op="decode", batch=4, new=1, lo=200, hi=1200, lens=6, heads=16, kv_heads=4, d=128,
             page=64),
        # Drafts of five tokens looked over at once, ragged lengths (none among them), small pages, d = 64.
        dict(name="decode_q4_drafts_d64", op="decode", batch=24, new=5, lo=0, hi=3000, lens=7, heads=12, kv_heads=4,
             d=64, page=16),
        # One sequence with a long context.
        dict(name="decode_q4_long", op="decode", batch=1, new=1, lo=131072, hi=131072, lens=8, heads=32, kv_heads=8,
             d=128, page=64),
        # A full batch of ragged sequences.
        dict(name="decode_q4_batch", op="decode", batch=64, new=1, lo=1024, hi=8192, lens=9, heads=32, kv_heads=8,
             d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "write_q4", "gather", "decode", "decode", "decode"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    lens = rng.randrange(10 ** 6)
    page = rng.choice([16, 32, 48, 64, 64, 128, 256])
    if op in ("append", "write_q4"):
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, batch=_log(rng, 1, min(64, tokens)), past=rng.choice([0, _log(rng, 1, 4000)]),
                    pad=rng.choice([0, 0, _log(rng, 1, 100)]), lens=lens, heads=heads, kv_heads=kv_heads, d=d,
                    rot=rng.choice([d, d, d // 2, 16, 48, 0]), interleaved=rng.random() < 0.4,
                    positions=_log(rng, 64, 131072), page=page)
    if op == "gather":
        hi = _log(rng, 2, 8192)
        return dict(op=op, batch=_log(rng, 1, 12), lo=int(hi * rng.uniform(0, 1)), hi=hi,
                    skip=rng.choice([0, _log(rng, 1, 1000)]), lens=lens, kv_heads=kv_heads, d=d, page=page)
    hi = _log(rng, 2, 65536)
    batch = _log(rng, 1, 64)
    while batch * hi > 64 * 4096:
        batch = max(1, batch // 2)
    return dict(op=op, batch=batch, new=rng.choice([1, 1, 1, 2, 4, 7]), lo=int(hi * rng.uniform(0, 1)), hi=hi,
                lens=lens, heads=heads, kv_heads=kv_heads, d=d, page=page)


def _lens(case):
    """The lengths of a case, which are its own: (tokens before, tokens that
    the operator handles) of each sequence."""
    r = random.Random(case["lens"])
    B = case["batch"]
    if case["op"] in ("append", "write_q4"):
        cuts = sorted(r.randint(0, case["tokens"] - B) for _ in range(B - 1))
        new = [b - a + 1 for a, b in zip([0] + cuts, cuts + [case["tokens"] - B])]
        return [r.randint(0, case["past"]) for _ in range(B)], new
    n = [r.randint(case["lo"], case["hi"]) for _ in range(B)]
    n[r.randrange(B)] = case["hi"]
    return [r.randint(0, case["skip"]) if case.get("skip") else 0 for _ in range(B)], n


def _q4_bytes(d):
    return d // 2 + d // GROUP * 4  # codes, scale and minimum of one row


def work(case):
    Hk, d = case["kv_heads"], case["d"]
    if case["op"] == "gather":
        n = sum(_lens(case)[1])
        return dict(bytes=n * Hk * 2 * (_q4_bytes(d) + 2 * d), flops=n * Hk * 4 * d)
    H = case["heads"]
    if case["op"] in ("append", "write_q4"):
        T, N = case["tokens"] + case["pad"], case["tokens"]
        rows = T * H * d * 4 + N * Hk * d * 4 + T * (case["rot"] * 4 + 8)  # q in and out, k and v in, tables
        if case["op"] == "append":
            return dict(bytes=rows + N * Hk * d * 4, flops=3 * case["rot"] * (T * H + N * Hk))
        return dict(bytes=rows + N * Hk * (4 * _q4_bytes(d) + 4 * d), flops=3 * case["rot"] * (T * H + N * Hk) +
                    N * Hk * 2 * d * 8)
    n = _lens(case)[1]
    new = case["new"]
    seen = sum(max(0, L - new + i + 1) for L in n for i in range(new))
    return dict(bytes=sum(n) * Hk * 2 * _q4_bytes(d) + case["batch"] * new * H * (4 * d + 4), flops=4 * d * H * seen)


# -------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g).to(BF16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _keys(g, *shape):
    """Keys as projections give them: channels of their own offset and width."""
    width = 0.3 + torch.rand(shape[-2:], device="cuda", generator=g)
    offset = torch.randn(shape[-2:], device="cuda", generator=g)
    return (torch.randn(*shape, device="cuda", generator=g) * width + offset).to(BF16)


def _pages(g, lens, page):
    """Pages of each sequence, scattered over a pool: (block table, pool size)."""
    count = [-(-n // page) for n in lens]
    pool = sum(count) + 3
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(len(lens), max(max(count), 1), dtype=torch.int32, device="cuda")
    at = _cu(count)
    for i, n in enumerate(count):
        table[i, :n] = order[at[i]:at[i + 1]]
    return table, pool


def _empty_q4(pool, Hk, page, d):
    codes = torch.zeros(2, pool, Hk, page, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, pool, Hk, page, d // GROUP, 2, dtype=BF16, device="cuda")
    return dict(k_codes=codes[0], k_scales=scales[0], v_codes=codes[1], v_scales=scales[1])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    Hk, d, page = case["kv_heads"], case["d"], case["page"]
    before, n = _lens(case)
    ends = [a + b for a, b in zip(before, n)]
    table, pool = _pages(g, ends, page)
    s = dict(case=case, block_table=table, scale=d ** -0.5, starts=_ints(before), cu=_ints(_cu(n)), seq_lens=_ints(n),
             max_len=max(max(n), 1))
    if case["op"] in ("append", "write_q4"):
        H, T, rot, span = case["heads"], case["tokens"] + case["pad"], case["rot"], case["positions"]
        # The fused projection's output: queries, keys and values of a token side by side.
        qkv = torch.cat((_normal(g, T, H, d), _keys(g, T, Hk, d), _normal(g, T, Hk, d)), 1)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:])
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
        angle = torch.arange(span, dtype=torch.float64, device="cuda")[:, None] * freq
        s.update(cos=angle.cos().float(), sin=angle.sin().float())
        at = torch.cat([torch.arange(a, a + b) for a, b in zip(before, n)]).cuda()
        seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n)).cuda()
        slots = table[seq, at // page] * page + (at % page).to(torch.int32)
        pad = torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")
        s.update(slots=torch.cat((slots.to(torch.int32), pad)), stored=case["tokens"],
                 positions=torch.cat((at % span, torch.zeros(case["pad"], device="cuda").long())).to(torch.int32),
                 q_out=torch.empty(T, H, d, dtype=BF16, device="cuda"))
        if case["op"] == "append":
            s.update(k_cache=_normal(g, pool, page, Hk, d), v_cache=_normal(g, pool, page, Hk, d))
            return s
        s.update(_empty_q4(pool, Hk, page, d))
    else:
        s.update(_empty_q4(pool, Hk, page, d))
        for name in "kv":
            rows = (_keys if name == "k" else _normal)(g, pool * page, Hk, d)
            codes, scales = _quantise(rows)
            s[name + "_codes"].copy_(codes.view(pool, page, Hk, -1).transpose(1, 2))
            s[name + "_scales"].copy_(scales.view(pool, page, Hk, -1, 2).transpose(1, 2))
        if case["op"] == "decode":
            H, new, B = case["heads"], case["new"], case["batch"]
            s.update(q=_normal(g, B, new, H, d), o=torch.empty(B, new, H, d, dtype=BF16, device="cuda"),
                     lse=torch.empty(B, new, H, device="cuda"))
            return s
    s.update(k_out=torch.empty(sum(n), Hk, d, dtype=BF16, device="cuda"),
             v_out=torch.empty(sum(n), Hk, d, dtype=BF16, device="cuda"))
    return s


# --------------------------------------------------------------- plain forms
def _rotate(x, s):
    """Every pair of the first rot elements turned by its token's angle, rounded to bf16."""
    at, rot = s["positions"].long(), s["case"]["rot"]
    c, n = s["cos"][at][:, None], s["sin"][at][:, None]
    x = x.float()
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((y, x[..., rot:]), -1).to(BF16)


def _quantise(x):
    """(codes, two a byte; scales and minima) of bf16 rows [..., d]."""
    x = x.float().unflatten(-1, (-1, GROUP))
    z, top = x.amin(-1), x.amax(-1)
    # Values next to a border between two codes: the quotients in 64 bits.
    s = ((top - z).double() / 15).float().to(BF16).float()
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    bad = ~torch.isfinite(s)
    s, z = s.masked_fill(bad, float("nan")), z.masked_fill(bad, float("nan"))
    t = (x - z[..., None]).double() / s[..., None].double()
    code = torch.where((s > 0)[..., None], t, torch.zeros_like(t)).round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.stack((s, z), -1).to(BF16)


def _values(codes, scales):
    """What rows of codes [..., d / 2] with scales [..., d / 64, 2] stand for, in 32 bits."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (scales[..., :1].float() * code + scales[..., 1:].float()).flatten(-2)


def _rows(s, name, slots):
    """The rows of the listed slots of a 4-bit cache, in 32 bits: [..., Hk, d]."""
    page = s["case"]["page"]
    block, at = slots // page, slots % page
    return _values(s[name + "_codes"][block, :, at], s[name + "_scales"][block, :, at])


def _plain_gather(s):
    total = s["k_out"].shape[0]
    row = torch.arange(total, device="cuda")
    seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    at = row - s["cu"].long()[seq] + s["starts"].long()[seq]
    page = s["case"]["page"]
    slots = s["block_table"].long()[seq, at // page] * page + at % page
    return _rows(s, "k", slots).to(BF16), _rows(s, "v", slots).to(BF16)


def _plain_append(s):
    q, k = _rotate(s["q"], s), _rotate(s["k"], s)
    slots = s["slots"][:s["stored"]].long()
    page = s["case"]["page"]
    block, at = slots // page, slots % page
    k, v = k[:s["stored"]], s["v"][:s["stored"]]
    if s["case"]["op"] == "append":
        s["k_cache"][block, at], s["v_cache"][block, at] = k, v
        return q, s["k_cache"], s["v_cache"]
    s["k_codes"][block, :, at], s["k_scales"][block, :, at] = _quantise(k)
    s["v_codes"][block, :, at], s["v_scales"][block, :, at] = _quantise(v)
    return q, *_plain_gather(s)


def _plain_decode(s):
    B, new, H, d = s["q"].shape
    Hk, page = s["case"]["kv_heads"], s["case"]["page"]
    q = s["q"].float().view(B, new, Hk, H // Hk, d).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, d)
    at = torch.arange(s["max_len"], device="cuda")
    slots = s["block_table"].long()[:, at // page] * page + at % page
    k, v = _rows(s, "k", slots), _rows(s, "v", slots)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    # Query i of a sequence sees the keys up to its own, the last query all of them.
    last = s["seq_lens"][:, None] - new + torch.arange(new, device="cuda")
    hidden = (at > last[..., None])[:, None, :, None].expand(-1, Hk, -1, H // Hk, -1)
    x = x.masked_fill(hidden.reshape(x.shape), NEG)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == NEG, 0.0))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + torch.log(z))[..., 0]
    o = o.view(B, Hk, new, H // Hk, d).permute(0, 2, 1, 3, 4).reshape(B, new, H, d)
    return o.to(BF16), lse.view(B, Hk, new, H // Hk).permute(0, 2, 1, 3).reshape(B, new, H).contiguous()


# ----------------------------------------------------------------------- run
def _own(s):
    from exact_io_aware_29_gb300 import binding as fa
    op = s["case"]["op"]
    cache = [s[name] for name in ("k_codes", "k_scales", "v_codes", "v_scales")] if op != "append" else []
    if op == "append":
        fa.fa_kv_append(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["positions"], s["slots"], s["q_out"],
                        s["k_cache"], s["v_cache"], s["case"]["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "write_q4":
        fa.fa_kv_append_q4(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["positions"], s["slots"], s["q_out"], *cache,
                           s["case"]["interleaved"])
        fa.fa_kv_gather_q4(*cache, s["block_table"], s["starts"], s["cu"], s["k_out"], s["v_out"])
        return s["q_out"], s["k_out"], s["v_out"]
    if op == "gather":
        fa.fa_kv_gather_q4(*cache, s["block_table"], s["starts"], s["cu"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if "ws" not in s:
        B, new, H, d = s["q"].shape
        size = fa.fa_decode_paged_q4_workspace_size(B, new, H, s["case"]["kv_heads"], d, s["max_len"])
        s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    fa.fa_decode_paged_q4(s["q"], *cache, s["o"], s["lse"], s["block_table"], s["seq_lens"], s["max_len"], s["scale"],
                          s["ws"])
    return s["o"], s["lse"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("append", "write_q4"):
        return _plain_append(state)
    return _plain_gather(state) if op == "gather" else _plain_decode(state)


# --------------------------------------------------------------------- exact
def _exact_rotated(x, s):
    half = s["case"]["rot"] // 2
    i = torch.arange(half, device="cuda")
    one, two = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + half)
    c, n = s["cos"].double()[s["positions"].long()][:, None], s["sin"].double()[s["positions"].long()][:, None]
    x = x.double()
    y = x.clone()
    y[..., one] = x[..., one] * c - x[..., two] * n
    y[..., two] = x[..., two] * c + x[..., one] * n
    return y


def _exact_held(x):
    """What the 4-bit cache holds in the place of bf16 rows [..., d]."""
    g = x.double().reshape(*x.shape[:-1], -1, GROUP)
    low, high = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    step = ((high - low) / 15).to(BF16).double()
    code = torch.where(step > 0, torch.round((g - low) / step), torch.zeros_like(g))
    return (low + step * code.clamp(max=15)).reshape(x.shape)


def _exact_slots(s, b, first, count):
    page = s["case"]["page"]
    t = torch.arange(first, first + count, device="cuda")
    return s["block_table"][b].long()[t // page], t % page


def _exact_read(s, name, b, first, count):
    """Tokens first.. of sequence b, as the cache holds them, in 64 bits: [count, Hk, d]."""
    block, at = _exact_slots(s, b, first, count)
    byte, sz = s[name + "_codes"][block, :, at], s[name + "_scales"][block, :, at].double()
    code = torch.empty(*byte.shape[:-1], 2 * byte.shape[-1], dtype=torch.float64, device="cuda")
    code[..., 0::2], code[..., 1::2] = byte % 16, byte // 16
    per = torch.repeat_interleave(sz, GROUP, -2)
    return per[..., 1] + per[..., 0] * code


def exact(case, seed):
    s = prepare(case, seed)
    before, n = _lens(case)
    if case["op"] in ("append", "write_q4"):
        q, k = _exact_rotated(s["q"], s), _exact_rotated(s["k"], s)
        v, N = s["v"].double(), case["tokens"]
        if case["op"] == "write_q4":
            return q, _exact_held(k[:N].to(BF16)), _exact_held(v[:N])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        t = 0
        for b, count in enumerate(n):
            where = _exact_slots(s, b, before[b], count)
            kc[where], vc[where] = k[t:t + count], v[t:t + count]
            t += count
        return q, kc, vc
    if case["op"] == "gather":
        return tuple(torch.cat([_exact_read(s, name, b, before[b], n[b]) for b in range(len(n))]) for name in "kv")
    B, new, H, d = s["q"].shape
    G = H // case["kv_heads"]
    o = torch.zeros(B, new, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, new, H), NEG, dtype=torch.float64, device="cuda")
    for b in range(B):
        k, v = _exact_read(s, "k", b, 0, n[b]), _exact_read(s, "v", b, 0, n[b])
        for i in range(new):
            seen = n[b] - new + i + 1
            for h in range(H if seen > 0 else 0):
                x = (k[:seen, h // G] @ s["q"][b, i, h].double()) * s["scale"]
                lse[b, i, h] = torch.logsumexp(x, 0)
                o[b, i, h] = torch.exp(x - lse[b, i, h]) @ v[:seen, h // G]
    return o, lse
