"""What is measured of the grouped-head operators: packed prompt attention
(forward, and forward with backward), query/key norms with the position
rotation (forward and backward), and decoding for a batch whose sequences
share long prefixes.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, each output rounded once) or, with ``own`` set, through the
package's binding, as a user's program calls it. ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
NEG = float("-inf")


# --------------------------------------------------------------------- cases
def listed():
    return [
        # A serving step that takes in many short prompts: latency and thin tiles.
        dict(name="prompt_short", op="prompt", batch=32, lo=1, hi=64, past=0, lens=1, heads=32, kv_heads=8, d=128),
        # Ragged prompts continued behind cached tokens, three query heads a key head.
        dict(name="prompt_ragged_d64", op="prompt", batch=9, lo=90, hi=2500, past=300, lens=2, heads=12, kv_heads=4,
             d=64),
        # Sixteen sequences of 512 to 8192 tokens, sixteen heads: the packed
        # batch that the benchmark times, with grouped heads.
        dict(name="prompt_long", op="prompt", batch=16, lo=512, hi=8192, past=0, lens=3, heads=16, kv_heads=4, d=128),
        # Training on a small ragged batch, seven query heads a key head.
        dict(name="train_ragged_d64", op="train", batch=7, lo=1, hi=900, past=0, lens=4, heads=14, kv_heads=2, d=64),
        # Training on packed documents of up to 4096 tokens.
        dict(name="train_packed", op="train", batch=8, lo=1024, hi=4096, past=0, lens=5, heads=16, kv_heads=4, d=128),
        # One generated token for each of a few sequences: latency.
        dict(name="norm_rope_step", op="rope", tokens=8, heads=32, kv_heads=8, d=128, rot=128, interleaved=False,
             positions=32768),
        # The queries and keys of a whole packed batch, read out of the fused projection.
        dict(name="norm_rope_prompt", op="rope", tokens=16384, heads=32, kv_heads=8, d=128, rot=128,
             interleaved=False, positions=32768),
        # The gradient on an odd number of tokens, with half of each head rotated, pairs side by side.
        dict(name="norm_rope_grad_odd", op="rope_grad", tokens=1001, heads=12, kv_heads=4, d=64, rot=32,
             interleaved=True, positions=5000),
        # The gradient on a training batch.
        dict(name="norm_rope_grad", op="rope_grad", tokens=16384, heads=32, kv_heads=8, d=128, rot=128,
             interleaved=False, positions=32768),
        # A few answers sampled from one prompt, just begun: latency.
        dict(name="decode_few", op="decode", prefixes=1, batch=4, plo=1000, phi=1000, slo=0, shi=200, lens=6, heads=16,
             kv_heads=4, d=128, page=64),
        # Several prompts of different lengths (one of them empty), full heads, d = 64.
        dict(name="decode_groups_d64", op="decode", prefixes=6, batch=40, plo=0, phi=4000, slo=1, shi=700, lens=7,
             heads=8, kv_heads=8, d=64, page=128),
        # A batch behind one long shared context.
        dict(name="decode_long_prefix", op="decode", prefixes=1, batch=64, plo=32768, phi=32768, slo=64, shi=1024,
             lens=8, heads=32, kv_heads=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "rope", "rope_grad", "decode", "decode"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    lens = rng.randrange(10 ** 6)
    if op in ("prompt", "train"):
        hi = _log(rng, 2, 4096 if op == "prompt" else 2048)
        batch = _log(rng, 1, 12)
        while heads > 1 and batch * heads * hi > 8 * 16 * 4096:
            batch = max(1, batch // 2)
            if batch == 1:
                break
        return dict(op=op, batch=batch, lo=max(0, int(hi * rng.uniform(-0.2, 0.9))), hi=hi,
                    past=rng.choice([0, 0, _log(rng, 1, 1000)]), lens=lens, heads=heads, kv_heads=kv_heads, d=d)
    if op in ("rope", "rope_grad"):
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=heads, kv_heads=kv_heads, d=d,
                    rot=rng.choice([d, d, d // 2, 16, 48]), interleaved=rng.random() < 0.4,
                    positions=_log(rng, 64, 131072))
    prefixes = rng.choice([1, 1, 2, 5])
    phi = _log(rng, 16, 20000)
    return dict(op=op, prefixes=prefixes, batch=prefixes * _log(rng, 1, 24), plo=int(phi * rng.uniform(0, 1)), phi=phi,
                slo=rng.choice([0, 1]), shi=_log(rng, 2, 1500), lens=lens, heads=heads, kv_heads=kv_heads, d=d,
                page=rng.choice([64, 64, 128, 256]))


def _lens(case):
    """The lengths of a case, which are its own: (queries, keys) of each packed
    sequence, or (sequences, prefix length) of each prefix and the suffix lengths."""
    r = random.Random(case["lens"])
    if case["op"] in ("prompt", "train"):
        lq = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
        lq[r.randrange(len(lq))] = case["hi"]
        return lq, [n + (r.randint(0, case["past"]) if case["past"] else 0) for n in lq]
    P, B = case["prefixes"], case["batch"]
    cuts = sorted(r.randint(0, B) for _ in range(P - 1))
    count = [b - a for a, b in zip([0] + cuts, cuts + [B])]
    plens = [r.randint(case["plo"], case["phi"]) for _ in range(P)]
    plens[0] = case["phi"]
    return count, plens, [r.randint(case["slo"], case["shi"]) for _ in range(B)]


def _pairs(case):
    """Visible (query, key) pairs of one head of a causal packed batch."""
    n = 0
    for a, b in zip(*_lens(case)):
        n += a * b - a * (a - 1) // 2  # lq <= lk here: row i sees lk - lq + i + 1 keys
    return n


def work(case):
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    if case["op"] in ("prompt", "train"):
        lq, lk = _lens(case)
        qo, kv = 2 * H * d * sum(lq), 2 * Hk * d * sum(lk)
        if case["op"] == "prompt":
            return dict(bytes=2 * qo + 2 * kv + 4 * H * sum(lq), flops=4 * d * H * _pairs(case))
        return dict(bytes=4 * qo + 4 * kv + 4 * H * sum(lq), flops=14 * d * H * _pairs(case))
    if case["op"] in ("rope", "rope_grad"):
        rows = case["tokens"] * (H + Hk)
        grad = case["op"] == "rope_grad"
        table = case["tokens"] * (case["rot"] * 4 + 4)  # a token's cosines, sines and position
        return dict(bytes=(3 if grad else 2) * rows * d * 2 + table + 4 * d + (8 * d if grad else 0),
                    flops=rows * d * (20 if grad else 8))
    count, plens, slens = _lens(case)
    keys = sum(p for p, n in zip(plens, count) if n) + sum(slens)
    seen = sum(p * n for p, n in zip(plens, count)) + sum(slens)
    B = case["batch"]
    return dict(bytes=4 * Hk * d * keys + 4 * B * H * d + 4 * B * H, flops=4 * d * H * seen)


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    s = dict(case=case, scale=d ** -0.5)
    if case["op"] in ("prompt", "train"):
        lq, lk = _lens(case)
        s.update(lq=lq, lk=lk, at_q=_cu(lq), at_k=_cu(lk), cu_q=_ints(_cu(lq)), cu_k=_ints(_cu(lk)))
        tq, tk = sum(lq), sum(lk)
        s.update(q=_normal(g, tq, H, d), k=_normal(g, tk, Hk, d), v=_normal(g, tk, Hk, d))
        s.update(o=torch.empty(tq, H, d, dtype=BF16, device="cuda"), lse=torch.empty(H, tq, device="cuda"))
        if case["op"] == "train":
            s["do"] = _normal(g, tq, H, d)
            s.update(dq=torch.empty_like(s["q"]), dk=torch.empty_like(s["k"]), dv=torch.empty_like(s["v"]))
        return s
    if case["op"] in ("rope", "rope_grad"):
        T, rot, n = case["tokens"], case["rot"], case["positions"]
        # The fused projection's output: queries, keys and values of a token side by side.
        qkv = _normal(g, T, (H + 2 * Hk) * d)
        s.update(qkv=qkv, q=qkv[:, :H * d].view(T, H, d), k=qkv[:, H * d:(H + Hk) * d].view(T, Hk, d))
        s.update(wq=(1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(BF16),
                 wk=(1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(BF16), eps=1e-6)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
        s.update(cos=angle.cos().float(), sin=angle.sin().float())
        first = torch.randint(0, n, (1,), device="cuda", generator=g)
        s["positions"] = ((first + torch.arange(T, device="cuda")) % n).to(torch.int32)
        s.update(yq=torch.empty(T, H, d, dtype=BF16, device="cuda"), yk=torch.empty(T, Hk, d, dtype=BF16, device="cuda"))
        if case["op"] == "rope_grad":
            s.update(gq=_normal(g, T, H, d), gk=_normal(g, T, Hk, d))
            s.update(dwq=torch.empty(d, device="cuda"), dwk=torch.empty(d, device="cuda"))
        return s
    count, plens, slens = _lens(case)
    page, B, P = case["page"], case["batch"], case["prefixes"]
    pages = [-(-n // page) for n in plens + slens]
    pool = sum(pages) + 3
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    mp, ms = max(max(pages[:P]), 1), max(max(pages[P:]), 1)
    ptab, stab = torch.zeros(P, mp, dtype=torch.int32, device="cuda"), torch.zeros(B, ms, dtype=torch.int32, device="cuda")
    at = _cu(pages)
    for i, n in enumerate(pages):
        (ptab[i] if i < P else stab[i - P])[:n] = order[at[i]:at[i + 1]]
    s.update(count=count, plens=plens, slens=slens, prefix_table=ptab, prefix_lens=_ints(plens), cu_seqs=_ints(_cu(count)),
             block_table=stab, seq_lens=_ints(slens), q=_normal(g, B, H, d), k=_normal(g, pool, page, Hk, d),
             v=_normal(g, pool, page, Hk, d), o=torch.empty(B, H, d, dtype=BF16, device="cuda"),
             lse=torch.empty(B, H, device="cuda"))
    return s


# --------------------------------------------------------------- plain forms
def _softmax(x):
    """(weights not yet divided, their sum, log of the sum of exp) over the last axis; rows of -inf give zeros."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == NEG, 0.0))
    z = p.sum(-1, keepdim=True)
    return p, z, m + torch.log(z)


def _attend(q, k, v, scale, shift):
    """One packed sequence: q [Lq, H, d], k and v [Lk, Hk, d] in 32 bits, bottom-right causal."""
    lq, H, d = q.shape
    lk, Hk, _ = k.shape
    qg = q.view(lq, Hk, H // Hk, d).permute(1, 2, 0, 3)
    x = torch.matmul(qg, k.permute(1, 2, 0)[:, None]) * scale
    hidden = torch.arange(lk, device=q.device) > torch.arange(lq, device=q.device)[:, None] + shift
    p, z, lse = _softmax(x.masked_fill_(hidden, NEG))
    p = p / torch.where(z > 0, z, torch.ones_like(z))
    return qg, p, torch.matmul(p, v.permute(1, 0, 2)[:, None]), lse[..., 0]


def _plain_packed(s, grad):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    (tq, H, d), Hk = q.shape, k.shape[1]
    o, lse = torch.zeros_like(q), torch.full((H, tq), NEG, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, (lq, lk) in enumerate(zip(s["lq"], s["lk"])):
        if lq == 0 or lk == 0:
            continue
        a, c = slice(s["at_q"][b], s["at_q"][b] + lq), slice(s["at_k"][b], s["at_k"][b] + lk)
        qg, p, og, lg = _attend(q[a], k[c], v[c], s["scale"], lk - lq)
        o[a] = og.permute(2, 0, 1, 3).reshape(lq, H, d)
        lse[:, a] = lg.reshape(H, lq)
        if grad:
            dog = s["do"][a].float().view(lq, Hk, H // Hk, d).permute(1, 2, 0, 3)
            dv[c] = torch.matmul(p.transpose(-1, -2), dog).sum(1).transpose(0, 1)
            dp = torch.matmul(dog, v[c].permute(1, 2, 0)[:, None])
            ds = p * (dp - (dog * og).sum(-1, keepdim=True)) * s["scale"]
            dq[a] = torch.matmul(ds, k[c].permute(1, 0, 2)[:, None]).permute(2, 0, 1, 3).reshape(lq, H, d)
            dk[c] = torch.matmul(ds.transpose(-1, -2), qg).sum(1).transpose(0, 1)
    if grad:
        return o.to(BF16), lse, dq.to(BF16), dk.to(BF16), dv.to(BF16)
    return o.to(BF16), lse


def _pair(x, rot, interleaved):
    """The two members of every rotated pair, and what is not rotated."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _unpair(a, b, rest, interleaved):
    both = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((both, rest), -1)


def _plain_rope(x, w, s):
    x, w = x.float(), w.float()
    u = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w
    at = s["positions"].long()
    c, n = s["cos"][at][:, None], s["sin"][at][:, None]
    rot, side = s["case"]["rot"], s["case"]["interleaved"]
    a, b, rest = _pair(u, rot, side)
    return _unpair(a * c - b * n, b * c + a * n, rest, side).to(BF16)


def _plain_rope_grad(x, w, g, s):
    x, w, g = x.float(), w.float(), g.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    at = s["positions"].long()
    c, n = s["cos"][at][:, None], s["sin"][at][:, None]
    rot, side = s["case"]["rot"], s["case"]["interleaved"]
    a, b, rest = _pair(g, rot, side)
    du = _unpair(a * c + b * n, b * c - a * n, rest, side)
    h = x * r
    dw = (du * h).sum((0, 1), dtype=torch.float64).float()
    dn = du * w
    return (r * (dn - h * (dn * h).mean(-1, keepdim=True))).to(BF16), dw


def _pages(pool, rows):
    """The tokens of the listed pages, in 32 bits: [rows, tokens, Hk, d]."""
    return pool[rows.long()].flatten(-4, -3).float()


def _plain_decode(s):
    q, H, Hk, d = s["q"].float(), s["case"]["heads"], s["case"]["kv_heads"], s["case"]["d"]
    B = q.shape[0]
    qg = q.view(B, Hk, H // Hk, d)
    # The sequences' own tokens, padded to the longest.
    k, v = _pages(s["k"], s["block_table"]), _pages(s["v"], s["block_table"])
    past = torch.arange(k.shape[1], device=q.device) >= s["seq_lens"][:, None]
    x = torch.matmul(qg, k.permute(0, 2, 3, 1)) * s["scale"]
    p, z, lse = _softmax(x.masked_fill(past[:, None, None], NEG))
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(z > 0, z, torch.ones_like(z))
    out, total = torch.empty_like(o), torch.empty_like(lse)
    b0 = 0
    for i, n in enumerate(s["count"]):
        b = slice(b0, b0 + n)
        b0 += n
        if n == 0:
            continue
        # The prefix once for all of its sequences, then the two parts joined by their sums.
        k, v = _pages(s["k"], s["prefix_table"][i])[:s["plens"][i]], _pages(s["v"], s["prefix_table"][i])[:s["plens"][i]]
        if s["plens"][i]:
            qp = qg[b].permute(1, 0, 2, 3).reshape(Hk, -1, d)
            p, z, lp = _softmax(torch.matmul(qp, k.permute(1, 2, 0)) * s["scale"])
            op = (torch.matmul(p, v.permute(1, 0, 2)) / z).view(Hk, n, H // Hk, d).transpose(0, 1)
            lp = lp.view(Hk, n, H // Hk, 1).transpose(0, 1)
        else:
            op, lp = torch.zeros_like(o[b]), torch.full_like(lse[b], NEG)
        m = torch.maximum(lp, lse[b])
        m0 = m.masked_fill(m == NEG, 0.0)
        wp, ws = torch.exp(lp - m0), torch.exp(lse[b] - m0)
        z = wp + ws
        out[b] = (wp * op + ws * o[b]) / torch.where(z > 0, z, torch.ones_like(z))
        total[b] = m + torch.log(z)
    return out.reshape(B, H, d).to(BF16), total.reshape(B, H)


# ----------------------------------------------------------------------- run
def _own(s):
    from exact_io_aware_29_gb300 import binding as fa
    op = s["case"]["op"]
    if op in ("prompt", "train"):
        mq, mk = max(s["lq"]), max(s["lk"])
        fa.fa_fwd_varlen_gqa(s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"], s["cu_k"], mq, mk, s["scale"], True)
        if op == "prompt":
            return s["o"], s["lse"]
        if "ws" not in s:
            s["ws"] = torch.empty(fa.fa_bwd_workspace_size(len(s["lq"]), s["case"]["heads"], mq, s["case"]["d"]),
                                  dtype=torch.uint8, device="cuda")
        fa.fa_bwd_varlen_gqa(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"], s["cu_q"],
                             s["cu_k"], mq, mk, s["scale"], True, s["ws"])
        return s["o"], s["lse"], s["dq"], s["dk"], s["dv"]
    if op == "rope":
        fa.fa_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], s["yq"], s["yk"],
                           s["eps"], s["case"]["interleaved"])
        return s["yq"], s["yk"]
    if op == "rope_grad":
        if "ws" not in s:
            n = fa.fa_qk_norm_rope_bwd_workspace_size(*s["q"].shape[:2], s["k"].shape[1], s["case"]["d"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        fa.fa_qk_norm_rope_bwd(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], s["gq"], s["gk"],
                               s["yq"], s["yk"], s["dwq"], s["dwk"], s["eps"], s["case"]["interleaved"], s["ws"])
        return s["yq"], s["yk"], s["dwq"], s["dwk"]
    c = s["case"]
    mc, mp, ml = max(s["count"]), max(max(s["plens"]), 1), max(max(s["slens"]), 1)
    if "ws" not in s:
        n = fa.fa_decode_shared_prefix_workspace_size(c["prefixes"], c["batch"], c["heads"], c["kv_heads"], c["d"], mc, mp, ml)
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    fa.fa_decode_shared_prefix(s["q"], s["k"], s["v"], s["o"], s["lse"], s["prefix_table"], s["prefix_lens"], s["cu_seqs"],
                               s["block_table"], s["seq_lens"], mc, mp, ml, s["scale"], s["ws"])
    return s["o"], s["lse"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("prompt", "train"):
        return _plain_packed(state, op == "train")
    if op == "rope":
        return _plain_rope(state["q"], state["wq"], state), _plain_rope(state["k"], state["wk"], state)
    if op == "rope_grad":
        dq, dwq = _plain_rope_grad(state["q"], state["wq"], state["gq"], state)
        dk, dwk = _plain_rope_grad(state["k"], state["wk"], state["gk"], state)
        return dq, dk, dwq, dwk
    return _plain_decode(state)


# --------------------------------------------------------------------- exact
def _exact_head(q, k, v, scale, first):
    """One head, rows whose last visible key is first + row (None: all keys), in 64 bits: P, O, log-sum-exp."""
    x = (q @ k.T) * scale
    if first is not None:
        x += torch.triu(torch.full_like(x, NEG), first + 1)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse.clamp_min(-1e300)[:, None])
    return p, p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    H, Hk, d = case["heads"], case["kv_heads"], case["d"]
    G = H // Hk
    if case["op"] in ("prompt", "train"):
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        o, lse = torch.zeros_like(q), torch.full((H, q.shape[0]), NEG, dtype=torch.float64, device="cuda")
        do = s["do"].double() if case["op"] == "train" else None
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b, (lq, lk) in enumerate(zip(s["lq"], s["lk"])):
            a, c = slice(s["at_q"][b], s["at_q"][b] + lq), slice(s["at_k"][b], s["at_k"][b] + lk)
            for h in range(H if lq and lk else 0):
                j = h // G
                p, o[a, h], lse[h, a] = _exact_head(q[a, h], k[c, j], v[c, j], s["scale"], lk - lq)
                if do is not None:
                    dv[c, j] += p.T @ do[a, h]
                    dp = do[a, h] @ v[c, j].T
                    ds = p * (dp - (dp * p).sum(1, keepdim=True))
                    dq[a, h] = s["scale"] * (ds @ k[c, j])
                    dk[c, j] += s["scale"] * (ds.T @ q[a, h])
        return (o, lse) if do is None else (o, lse, dq, dk, dv)
    if case["op"] in ("rope", "rope_grad"):
        grads, sums = [], []
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda")
        one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        c, n = s["cos"].double()[s["positions"].long()][:, None], s["sin"].double()[s["positions"].long()][:, None]
        for name in "qk":
            x = s[name].double().requires_grad_()
            w = s["w" + name].double().requires_grad_()
            u = w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + s["eps"])
            y = u.clone()
            y[..., one] = u[..., one] * c - u[..., two] * n
            y[..., two] = u[..., two] * c + u[..., one] * n
            if case["op"] == "rope":
                grads.append(y.detach())
            else:
                dx, dw = torch.autograd.grad(y, (x, w), s["g" + name].double())
                grads.append(dx)
                sums.append(dw)
        return tuple(grads + sums)
    page = case["page"]
    o = torch.zeros(case["batch"], H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], H), NEG, dtype=torch.float64, device="cuda")
    flat_k, flat_v = s["k"].view(-1, Hk, d), s["v"].view(-1, Hk, d)
    b = 0
    for i, n in enumerate(s["count"]):
        def slots(table, count):
            t = torch.arange(count, device="cuda")
            return table.long()[t // page] * page + t % page
        own_prefix = slots(s["prefix_table"][i], s["plens"][i])
        for b in range(b, b + n):
            at = torch.cat((own_prefix, slots(s["block_table"][b], s["slens"][b])))
            if at.numel():
                kk, vv = flat_k[at].double(), flat_v[at].double()
                x = torch.einsum("jgd,ljd->jgl", s["q"][b].double().view(Hk, G, d), kk) * s["scale"]
                lse[b] = torch.logsumexp(x, -1).reshape(H)
                o[b] = torch.einsum("jgl,ljd->jgd", torch.softmax(x, -1), vv).reshape(H, d)
        b = b + 1 if n else b
    return o, lse
