"""Measured cases of the operators around a served batch whose sequences share a prefix.

Three operators: new tokens appended to the paged cache (norm and rotation of
queries and keys, and the cache's write, in one pass), pages copied to pages
where sequences fork, and the attention of new tokens over the cache where
groups of sequences hold the same prefix in the same pages, computed once for
all of a group. `run` with own = False computes them in elementary torch
operations in 32 bits; with own = True it makes the library's calls.
"""
import math

import torch

own = False

BF16, F32, F64, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


# --------------------------------------------------------------------- cases
def _append(name, R, tokens, kv, hq, hkv, d, page, e4m3, rot, inter, norm, wtype, scaled, given):
    return dict(name=name, op="append", R=R, tokens=tokens, kv=kv, hq=hq, hkv=hkv, d=d, page=page, e4m3=e4m3, rot=rot,
                inter=inter, norm=norm, wtype=wtype, scaled=scaled, given=given)


def _copy(name, n, hkv, d, page, e4m3):
    return dict(name=name, op="copy", n=n, hkv=hkv, d=d, page=page, e4m3=e4m3)


def _shared(name, S, R, tokens, prefix, more, hq, hkv, d, page, e4m3, causal=True):
    return dict(name=name, op="shared", S=S, R=R, tokens=tokens, prefix=prefix, more=more, hq=hq, hkv=hkv, d=d, page=page,
                e4m3=e4m3, causal=causal)


def listed():
    return [
        # a decoding step of 64 sequences: one token each, between the projection and the attention: latency
        _append("append_step_e4m3", 64, 64, 2048, 32, 8, 128, 16, True, 128, False, True, "f32", True, False),
        # a small model's packed batch: part of the head rotated, interleaved pairs, no norm, odd lengths, positions given
        _append("append_small", 3, 1037, 700, 2, 2, 64, 32, False, 32, True, False, "f32", False, True),
        # chunks of four long prompts into a quantised cache
        _append("append_chunk_e4m3", 4, 8192, 12288, 32, 8, 128, 64, True, 128, False, True, "bf16", False, False),
        # two prompts of 16K tokens and wide groups: bandwidth
        _append("append_32k", 2, 32768, 16384, 64, 8, 128, 64, False, 128, True, True, "f32", True, False),
        # a prompt's last, partly filled page, copied for each of eight responses: latency
        _copy("copy_fork", 8, 8, 128, 64, False),
        # the pages of beams that change places
        _copy("copy_beams_e4m3", 4096, 8, 128, 64, True),
        # the smallest call: the first tokens of two responses to one short question
        _shared("shared_two", 1, 2, 2, 1021, 40, 32, 8, 128, 16, False),
        # a step of eight responses to one question, lengths as the share-question data have them
        _shared("shared_question", 1, 8, 8, 2048, 1024, 32, 8, 128, 64, False),
        # a step of six questions with responses of their own, small heads, a quantised cache
        _shared("shared_groups_e4m3", 6, 48, 48, 4096, 700, 16, 2, 64, 32, True),
        # a step of 64 samples of a long document's summary over a quantised cache
        _shared("shared_step_e4m3", 1, 64, 64, 16384, 1024, 32, 8, 128, 64, True),
        # a step of 128 samples behind a 32K prompt, wide groups: bandwidth and matrix rate
        _shared("shared_step_32k", 1, 128, 128, 32768, 1024, 64, 8, 128, 64, False),
        # chunks of 32 short questions, 20 to 60 tokens each, behind one system prompt
        _shared("shared_chunks", 1, 32, 1279, 8192, 64, 32, 8, 128, 64, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "append", "copy", "shared", "shared", "shared", "shared"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 8])
    group = rng.choice([1, 2, 4, 5, 8, 64] if hkv == 1 else [1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    e4m3 = rng.random() < 0.5
    if op == "append":
        R = _log(rng, 1, 64)
        tokens = max(1, _log(rng, R, min(32768, 32768 * 80 * 128 // (hkv * (group + 2) * d))))
        kv = max(-(-tokens // R), _log(rng, 1, 65536 // R))
        rot = rng.choice([0, d, d, d // 2, 16])
        return dict(op="append", R=R, tokens=tokens, kv=kv, hq=hkv * group, hkv=hkv, d=d, page=page, e4m3=e4m3, rot=rot,
                    inter=rng.random() < 0.5, norm=rng.random() < 0.7, wtype=rng.choice(["f32", "bf16"]),
                    scaled=rng.random() < 0.5, given=rng.random() < 0.3)
    if op == "copy":
        return dict(op="copy", n=_log(rng, 1, min(8192, (1 << (28 if e4m3 else 27)) // (hkv * page * d))), hkv=hkv, d=d, page=page, e4m3=e4m3)
    S = rng.choice([1, 1, 1, _log(rng, 1, 8)])
    R = S * _log(rng, 1, 128 // S) + (rng.randrange(S) if S < 8 else 0)
    prefix = _log(rng, 1, 32768 // S)
    more = _log(rng, 1, 2048)
    # a token a sequence, a few (drafts), or chunks; the plain form's scores bound the product
    most = max(1, (1 << 34) // ((prefix + more) * hkv * group * R * d))
    tokens = R * max(1, min(most, rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 17, 256)])))
    if tokens > R:
        tokens -= rng.randrange(R)
    return dict(op="shared", S=S, R=R, tokens=tokens, prefix=prefix, more=more, hq=hkv * group, hkv=hkv, d=d, page=page,
                e4m3=e4m3, causal=rng.random() < 0.85)


# -------------------------------------------------------------------- inputs
def _new_and_keys(R, tokens, kv):
    """New tokens and keys of each sequence, from the case alone: ragged, the longest of
    them kv keys, each at least its new tokens."""
    part = torch.rand(R, generator=torch.Generator().manual_seed(1000003 * R + kv)).tolist()
    new = [tokens // R + (1 if r < tokens % R else 0) for r in range(R)]
    low = 0.25 if R > 1 else 1.0
    keys = [max(new[r], int(round(kv * (low + (1 - low) * part[r])))) for r in range(R)]
    keys[0] = max(new[0], kv)
    return new, keys


def _groups(case):
    """New tokens and keys of each sequence, first sequence and shared keys of each group."""
    S, R, tokens = case["S"], case["R"], case["tokens"]
    g = torch.Generator().manual_seed(1000003 * R + case["prefix"])
    part = torch.rand(S, generator=g).tolist()
    low = 0.25 if S > 1 else 1.0
    prefix = [max(1, int(round(case["prefix"] * (low + (1 - low) * x)))) for x in part]
    prefix[0] = case["prefix"]
    # group sizes between half and twice their mean
    w = [1 + 2 * x for x in torch.rand(S, generator=g).tolist()]
    first = [0]
    for s in range(S):
        left = S - 1 - s  # groups still to come hold a sequence each
        n = R - first[-1] if not left else max(1, min(R - first[-1] - left, int(round(R * w[s] / sum(w)))))
        first.append(first[-1] + n)
    if tokens >= 2 * R:  # chunks of between half and one and a half times their mean
        w = [0.5 + x for x in torch.rand(R, generator=g).tolist()]
        new = [max(1, int(tokens * x / sum(w))) for x in w]
        new[0] += tokens - sum(new)
    else:
        new = [tokens // R + (1 if r < tokens % R else 0) for r in range(R)]
    part = torch.rand(R, generator=g).tolist()
    keys = [0] * R
    for s in range(S):
        for r in range(first[s], first[s + 1]):
            keys[r] = prefix[s] + max(new[r], int(round(case["more"] * part[r])))
    return new, keys, first, prefix


def _freqs(rot, scaled):
    """Inverse frequencies and the factor of cos and sin: plain, or blended between the
    plain and the 8 times slower ones by the turns a pair makes in 4096 positions."""
    i = torch.arange(rot // 2, dtype=F64)
    f = 10000.0 ** (-2.0 * i / rot)
    if not scaled:
        return f.to(F32), 1.0
    where = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(0.0, math.floor(where(32.0))), min(rot - 1.0, math.ceil(where(1.0)))
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return (f / 8.0 * ramp + f * (1 - ramp)).to(F32), 0.1 * math.log(8.0) + 1.0


def _randn(shape, gen, dtype=BF16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=F32).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(s, n_pages, gen):
    """The cache's pages: random rows, with one scale each where they are e4m3, as a
    write leaves them: largest value in (224, 448]."""
    for x in ("kc", "vc"):
        c = _randn((n_pages, s["hkv"], s["page"], s["d"]), gen)
        if s["e4m3"]:
            top = c.abs().amax(-1, keepdim=True).to(F32)
            e = torch.ceil(torch.log2(top / 448.0))
            s[x] = (c.to(F32) * torch.exp2(-e)).to(E4M3)
            s[x + "_exp"] = (e.squeeze(-1) + 127).to(torch.uint8)
        else:
            s[x], s[x + "_exp"] = c, None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    hq, hkv, d, page = case.get("hq"), case["hkv"], case["d"], case["page"]
    up = lambda x: -(-x // page)  # noqa: E731
    if case["op"] == "copy":
        # pages in an order of their own: the first half of them to the second
        order = torch.randperm(2 * case["n"] + 3, generator=gen, device="cuda").to(torch.int32)
        s["src"], s["dst"] = order[: case["n"]].contiguous(), order[case["n"]:2 * case["n"]].contiguous()
        _pages(s, 2 * case["n"] + 3, gen)
    elif case["op"] == "append":
        R = case["R"]
        new, keys = _new_and_keys(R, case["tokens"], case["kv"])
        order = torch.randperm(sum(up(x) for x in keys) + 3, generator=gen, device="cuda").to(torch.int32)
        s["table"] = torch.full((R, max(up(x) for x in keys)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for r in range(R):
            s["table"][r, :up(keys[r])] = order[at:at + up(keys[r])]
            at += up(keys[r])
        _pages(s, order.numel(), gen)
        # the fused projection's output, and views of it
        qkv = _randn((case["tokens"], hq + 2 * hkv, d), gen)
        s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], 1)
        s["freq"], s["rot_scale"] = None, 1.0
        if case["rot"]:
            f, s["rot_scale"] = _freqs(case["rot"], case["scaled"])
            s["freq"] = f.cuda()
        # positions that are not the places in the cache: a document's own, far into a context
        s["pos"] = torch.randint(0, 131072, (case["tokens"],), generator=gen, device="cuda").to(torch.int32) if case["given"] else None
        wt = F32 if case["wtype"] == "f32" else BF16
        s["wq"], s["wk"] = ((1 + 0.2 * _randn((d,), gen, F32)).to(wt) if case["norm"] else None for _ in range(2))
    else:
        S, R = case["S"], case["R"]
        new, keys, first, prefix = _groups(case)
        s["groups"], s["new"], s["keys"] = (first, prefix), new, keys
        whole = [x // page for x in prefix]  # pages that a group's sequences share
        n_pages = sum(whole) + sum(up(keys[r]) - whole[g] for g in range(S) for r in range(first[g], first[g + 1])) + 3
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        s["table"] = torch.full((R, max(up(x) for x in keys)), -1, dtype=torch.int32, device="cuda")
        _pages(s, n_pages, gen)
        at = 0
        for g in range(S):
            lo, hi, w = first[g], first[g + 1], whole[g]
            s["table"][lo:hi, :w] = order[at:at + w]
            at += w
            for r in range(lo, hi):
                s["table"][r, w:up(keys[r])] = order[at:at + up(keys[r]) - w]
                at += up(keys[r]) - w
            if prefix[g] % page and hi > lo + 1:
                # the prefix's last, partly filled page: each sequence has a copy
                own_pages = s["table"][lo:hi, w].long()
                for x in ("kc", "vc", "kc_exp", "vc_exp"):
                    if s[x] is not None:
                        b = s[x] if s[x].dtype != E4M3 else s[x].view(torch.uint8)
                        b[own_pages[1:], :, :prefix[g] % page] = b[own_pages[0], :, :prefix[g] % page]
        s["q"] = _randn((case["tokens"], hq, d), gen)
        s["scale"] = d ** -0.5
        s["seq_off"], s["prefix_len"] = _i32(first), _i32(prefix)
    if case["op"] != "copy":
        s["q_off"] = _i32([sum(new[:r]) for r in range(len(new) + 1)])
        s["kv_len"] = _i32(keys)
    if own:
        # the handles a serving program keeps: checked views of the tensors above, nothing computed
        import mask_aware_sparse_gb300 as fm

        s["cache"] = fm.KVCache(s["kc"], s["vc"], s["kc_exp"], s["vc_exp"])
        if case["op"] != "copy":
            s["batch"] = fm.PagedBatch(s["q_off"], s["kv_len"], s["table"])
        if case["op"] == "shared":
            s["shared"] = fm.SharedPrefix(s["seq_off"], s["prefix_len"])
    return s


# --------------------------------------------------------------- plain forms
def _cache_of(s):
    """The cache: its rows, and the scales as the powers of two that their bytes stand for."""
    return [s[x].view(E8M0) if x.endswith("exp") else s[x] for x in ("kc", "kc_exp", "vc", "vc_exp") if s[x] is not None]


def _sequence_of_tokens(off, T):
    """The sequence of each of T tokens, and its number among the sequence's new ones."""
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return r, t - off[r]


def _plain_append(s):
    n, rot, inter = s["q_off"].long(), s["rot"], s["inter"]
    r, a = _sequence_of_tokens(n, s["tokens"])
    place = s["kv_len"].long()[r] - (n[r + 1] - n[r]) + a
    page, slot = s["table"].long()[r, place // s["page"]], place % s["page"]
    if rot:
        turn = (place if s["pos"] is None else s["pos"]).to(F64)[:, None] * s["freq"].to(F64)  # far positions: 64 bits
        cos, sin = ((f(turn).to(F32) * s["rot_scale"])[:, None] for f in (torch.cos, torch.sin))

    def turned(x, w):
        x = x.to(F32)
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(F32)
        if not rot:
            return x
        h = x[..., :rot]
        p, q = (h[..., 0::2], h[..., 1::2]) if inter else (h[..., :rot // 2], h[..., rot // 2:])
        p, q = p * cos - q * sin, p * sin + q * cos
        h = torch.stack((p, q), -1).flatten(-2) if inter else torch.cat((p, q), -1)
        return torch.cat((h, x[..., rot:]), -1)

    for x, c in ((turned(s["k"], s["wk"]), "kc"), (s["v"].to(F32), "vc")):
        if s["e4m3"]:
            top = x.abs().amax(-1, keepdim=True)
            m, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
            e = (e - 9 + (m > 0.875)).clamp(min=-126)
            e = torch.where(top > 0, e, torch.full_like(e, -126))
            s[c + "_exp"][page, :, slot] = (e.squeeze(-1) + 127).to(torch.uint8)
            s[c].view(torch.uint8)[page, :, slot] = torch.ldexp(x, -e).to(E4M3).view(torch.uint8)
        else:
            s[c][page, :, slot] = x.to(BF16)
    return [turned(s["q"], s["wq"]).to(BF16)] + _cache_of(s)


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for x in ("kc", "vc", "kc_exp", "vc_exp"):
        if s[x] is not None:
            b = s[x].view(torch.uint8) if s["e4m3"] else s[x]
            b[dst] = b[src]
    return _cache_of(s)


def _values(s, x, pages):
    """Rows of whole pages (..., n) as 32-bit values (..., H_kv, n * page, d)."""
    c = s[x][pages].to(F32)
    if s["e4m3"]:
        c = c * torch.exp2(s[x + "_exp"][pages].to(F32) - 127)[..., None]
    return c.transpose(-4, -3).flatten(-3, -2)


def _part(s, q, rows, pages, see):
    """Unnormalised attention of padded rows: q (T, H_q, d), rows (B, n) token numbers, pages
    (B, m), see (B, n, m * page). Largest score, sum of exp and of exp times the values."""
    B, n = rows.shape
    G = s["hq"] // s["hkv"]
    x = q[rows].view(B, n, s["hkv"], G, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)  # (B, H_kv, n * G, d)
    held = see.any(1)[:, None, :, None]
    sc = torch.matmul(x, _values(s, "kc", pages).masked_fill_(~held, 0.0).transpose(-1, -2)).mul_(s["scale"])
    sc.masked_fill_(~see.repeat_interleave(G, 1)[:, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = sc.sub_(top.clamp(min=-1e30)).exp_()
    back = lambda x: x.view(B, s["hkv"], n, G, -1).permute(0, 2, 1, 3, 4).reshape(B, n, s["hq"], -1)  # noqa: E731
    return back(top), back(p.sum(-1, keepdim=True)), back(torch.matmul(p, _values(s, "vc", pages).masked_fill_(~held, 0.0)))


def _plain_shared(s):
    page, T, (first, prefix) = s["page"], s["tokens"], s["groups"]
    q, q_off, kv_len, table = s["q"].to(F32), s["q_off"].long(), s["kv_len"].long(), s["table"].long().clamp(min=0)
    seq_off, whole = s["seq_off"].long(), s["prefix_len"].long() // page  # pages that are shared
    r, a = _sequence_of_tokens(q_off, T)
    g, _ = _sequence_of_tokens(seq_off, s["R"])  # of each sequence
    # the groups' new tokens over the shared pages
    t0 = q_off[seq_off]
    most = max(sum(s["new"][first[i]:first[i + 1]]) for i in range(s["S"]))
    wide = max(1, max(prefix) // page)
    rows = (t0[:-1, None] + torch.arange(most, device="cuda")).clamp(max=T - 1)
    j = torch.arange(wide * page, device="cuda")
    see = (j < (whole * page)[:, None])[:, None].expand(-1, most, -1)
    pages = table[seq_off[:-1], :wide]
    one = [x[g[r], torch.arange(T, device="cuda") - t0[g[r]]] for x in _part(s, q, rows, pages, see)]
    # each sequence's new tokens over its other pages
    most, n = max(s["new"]), q_off[1:] - q_off[:-1]
    wide = max(-(-k // page) - prefix[i] // page for i in range(s["S"]) for k in s["keys"][first[i]:first[i + 1]])
    rows = (q_off[:-1, None] + torch.arange(most, device="cuda")).clamp(max=T - 1)
    col = whole[g][:, None] + torch.arange(wide, device="cuda")
    pages = table.gather(1, col.clamp(max=table.shape[1] - 1))
    j = ((whole[g] * page)[:, None] + torch.arange(wide * page, device="cuda"))[:, None]
    see = j < kv_len[:, None, None]
    if s["causal"]:
        see = see & (j <= (kv_len - n)[:, None, None] + torch.arange(most, device="cuda")[:, None])
    two = [x[r, a] for x in _part(s, q, rows, pages, see.expand(-1, most, -1))]
    top = torch.maximum(one[0], two[0])
    w1, w2 = (torch.exp(x[0] - top.clamp(min=-1e30)) for x in (one, two))
    total = w1 * one[1] + w2 * two[1]
    o = (w1 * one[2] + w2 * two[2]) / total.clamp(min=1e-30)
    return [o.to(BF16), (top + torch.log(total)).squeeze(-1)]


def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "copy": _plain_copy, "shared": _plain_shared}[s["op"]](s)
    import mask_aware_sparse_gb300 as fm

    if s["op"] == "append":
        q = fm.fm_cache_append(s["q"], s["k"], s["v"], s["cache"], s["batch"], positions=s["pos"], inv_freq=s["freq"],
                               interleaved=s["inter"], rot_scale=s["rot_scale"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
        return [q] + _cache_of(s)
    if s["op"] == "copy":
        fm.fm_cache_copy(s["cache"], s["src"], s["dst"])
        return _cache_of(s)
    return list(fm.fm_attn_shared(s["q"], s["cache"], s["batch"], s["shared"], scale=s["scale"], causal=s["causal"]))


# ---------------------------------------------------------------------- work
def work(case):
    hkv, d = case["hkv"], case["d"]
    row = hkv * (d + 1 if case["e4m3"] else 2 * d)  # a cached token's keys, or its values
    if case["op"] == "append":
        T, hq = case["tokens"], case["hq"]
        return {"bytes": T * ((hq * 2 + hkv * 2) * d * 2 + 2 * row), "flops": T * (hq + hkv) * d * 8}
    if case["op"] == "copy":
        return {"bytes": 4 * case["n"] * case["page"] * row, "flops": 0}
    new, keys, first, prefix = _groups(case)
    page, cols, pairs = case["page"], 0, 0
    for g in range(case["S"]):
        w = prefix[g] // page * page
        cols += w
        for r in range(first[g], first[g + 1]):
            cols += keys[r] - w
            pairs += new[r] * keys[r] - (new[r] * (new[r] - 1) // 2 if case["causal"] else 0)
    return {"bytes": 2 * cols * row + case["tokens"] * case["hq"] * (d * 4 + 4), "flops": 4 * pairs * case["hq"] * d}


# --------------------------------------------------------------------- exact
def _exact_append(s):
    """Token places by counting, the rotation as a complex product, in 64 bits."""
    T, rot = s["tokens"], s["rot"]
    q_off, keys = s["q_off"].tolist(), s["kv_len"].tolist()
    seq = [r for r in range(s["R"]) for _ in range(q_off[r + 1] - q_off[r])]
    place = torch.tensor([keys[r] - q_off[r + 1] + t for t, r in enumerate(seq)], device="cuda")
    pages = s["table"][torch.tensor(seq, device="cuda"), place // s["page"]].long()

    def f(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
        if not rot:
            return x
        theta = (place if s["pos"] is None else s["pos"]).double()[:, None, None] * s["freq"].double()
        z = torch.polar(torch.full_like(theta, s["rot_scale"]), theta)
        head = x[..., :rot]
        if s["inter"]:
            c = torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous())
            head = torch.view_as_real(c * z).flatten(-2)
        else:
            c = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * z
            head = torch.cat((c.real, c.imag), -1)
        return torch.cat((head, x[..., rot:]), -1)

    out = [f(s["q"], s["wq"])]
    for x, c in ((f(s["k"], s["wk"]), "kc"), (s["v"].double(), "vc")):
        if s["e4m3"]:
            return out + [None] * 4  # rounded to the cache's type by definition
        rows = s[c].double()
        rows[pages, :, place % s["page"]] = x
        out.append(rows)
    return out


def _exact_shared(s):
    """Sequence by sequence over its own page table, keys gathered page by page."""
    out = torch.zeros(s["tokens"], s["hq"], s["d"], dtype=F64, device="cuda")
    lse = torch.full((s["tokens"], s["hq"]), -math.inf, dtype=F64, device="cuda")
    G, at = s["hq"] // s["hkv"], 0
    for r, (n, L) in enumerate(zip(s["new"], s["keys"])):
        pages = s["table"][r, : -(-L // s["page"])].long()
        for h in range(s["hkv"]):
            kv = []
            for c in ("kc", "vc"):
                x = s[c][pages, h].double()
                if s["e4m3"]:
                    x = x * torch.pow(2.0, s[c + "_exp"][pages, h].double() - 127)[..., None]
                kv.append(x.reshape(-1, s["d"])[:L])
            w = torch.einsum("agd,jd->agj", s["q"][at:at + n, h * G:(h + 1) * G].double(), kv[0]) * s["scale"]
            if s["causal"]:
                ahead = torch.arange(L, device="cuda") > torch.arange(L - n, L, device="cuda")[:, None]
                w = w.masked_fill(ahead[:, None, :], -math.inf)
            lse[at:at + n, h * G:(h + 1) * G] = torch.logsumexp(w, -1)
            out[at:at + n, h * G:(h + 1) * G] = torch.einsum("agj,jd->agd", torch.softmax(w, -1), kv[1])
        at += n
    return [out, lse]


def _exact_copy(s):
    rows = [x.double() for x in _cache_of(s)]
    to = dict(zip(s["dst"].tolist(), s["src"].tolist()))
    of = torch.tensor([to.get(i, i) for i in range(rows[0].shape[0])], device="cuda")
    return [x[of] for x in rows]


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "copy": _exact_copy, "shared": _exact_shared}[case["op"]](s)
