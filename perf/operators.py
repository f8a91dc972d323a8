"""Measured cases of the operators around a served or trained attention layer.

Three operators: the norm and rotation of queries and keys in one pass (with
its backward), the paged key / value cache as it is written and read back, and
the attention of new tokens over that cache. `run` with own = False computes
them in elementary torch operations in 32 bits; with own = True it makes the
library's calls.
"""
import math

import torch

own = False

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn


# --------------------------------------------------------------------- cases
def _qk(name, B, N, hq, hkv, d, rot, inter, norm, wtype, scaled, far, bwd):
    return dict(name=name, op="qk", B=B, N=N, hq=hq, hkv=hkv, d=d, rot=rot, inter=inter, norm=norm, wtype=wtype,
                scaled=scaled, far=far, bwd=bwd)


def _cache(name, op, R, tokens, kv, hkv, d, page, e4m3):
    return dict(name=name, op=op, R=R, tokens=tokens, kv=kv, hkv=hkv, d=d, page=page, e4m3=e4m3)


def _attn(name, R, tokens, kv, hq, hkv, d, page, e4m3, causal=True, window=0, sinks=0):
    return dict(name=name, op="attn", R=R, tokens=tokens, kv=kv, hq=hq, hkv=hkv, d=d, page=page, e4m3=e4m3,
                causal=causal, window=window, sinks=sinks)


def listed():
    return [
        # one decoding step of eight sequences far into a long context: latency
        _qk("qk_step", 8, 1, 32, 8, 128, 128, False, True, "f32", True, 131072, False),
        # a small model's packed batch: part of the head rotated, interleaved pairs, no norm, odd length, both ways
        _qk("qk_small_both_ways", 3, 1037, 2, 2, 64, 32, True, False, "f32", False, 1037, True),
        # a training step on the 8K document packing: norms with their weights' gradients, both ways
        _qk("qk_train_8k", 1, 8192, 32, 8, 128, 128, False, True, "bf16", False, 8192, True),
        # the forward of a 64K packing with wide heads
        _qk("qk_forward_64k", 1, 65536, 64, 8, 128, 128, True, True, "f32", True, 65536, False),
        # the new keys and values of one decoding step of 64 sequences
        _cache("cache_step_e4m3", "write", 64, 64, 2048, 8, 128, 16, True),
        # the new keys and values of long prompts' chunks
        _cache("cache_chunk_e4m3", "write", 4, 8192, 12288, 8, 128, 64, True),
        # a cache read back as packed documents, for scoring with gradients
        _cache("cache_read_e4m3", "read", 4, 0, 16384, 8, 128, 64, True),
        # the smallest call: one new token of one short sequence
        _attn("attn_one_token", 1, 1, 1021, 32, 8, 128, 16, False),
        # one decoding step of 32 sequences of ragged lengths over a quantised cache: bandwidth
        _attn("attn_step_e4m3", 32, 32, 16384, 32, 8, 128, 64, True),
        # one decoding step of a model trained with a sliding window and sinks
        _attn("attn_step_window", 8, 8, 65536, 64, 8, 128, 32, False, window=4096, sinks=4),
        # ragged chunks of a few hundred tokens over a quantised cache, small heads
        _attn("attn_chunks_e4m3", 5, 1111, 3000, 16, 2, 64, 32, True),
        # a chunk of a long prompt: matrix rate
        _attn("attn_chunk_32k", 1, 2048, 32768, 32, 8, 128, 64, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk", "write", "read", "attn", "attn", "attn"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 8])
    group = rng.choice([1, 2, 4, 5, 8, 64] if hkv == 1 else [1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "qk":
        B = _log(rng, 1, 8)
        N = _log(rng, 1, 65536 * 72 * 128 // (B * hkv * (group + 1) * d * 8))
        rot = rng.choice([d, d, d // 2, 16])
        return dict(op="qk", B=B, N=N, hq=hkv * group, hkv=hkv, d=d, rot=rot, inter=rng.random() < 0.5,
                    norm=rng.random() < 0.7, wtype=rng.choice(["f32", "bf16"]), scaled=rng.random() < 0.5,
                    far=_log(rng, max(N, 2), 1 << 20 if N < 1 << 20 else N), bwd=rng.random() < 0.5)
    R = _log(rng, 1, 64)
    if op in ("write", "read"):
        kv = _log(rng, 1, 65536 // R)
        return dict(op=op, R=R, tokens=min(R * kv, _log(rng, R, 8192 + R)) if op == "write" else 0, kv=kv, hkv=hkv,
                    d=d, page=page, e4m3=rng.random() < 0.7)
    kv = _log(rng, 1, 262144 // R)
    # few tokens a sequence (steps, drafts) or a chunk; the plain form's scores bound the product
    most = max(1, min(kv, 1 << 30, 2048 * 32768 * 32 // (kv * hkv * group * R * 2)))
    tokens = R * max(1, min(most, rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 2048)])))
    if tokens > R:
        tokens -= rng.randrange(R)
    causal = rng.random() < 0.8
    window = _log(rng, 1, max(2, kv)) if causal and rng.random() < 0.3 else 0
    return dict(op="attn", R=R, tokens=tokens, kv=kv, hq=hkv * group, hkv=hkv, d=d, page=page,
                e4m3=rng.random() < 0.5, causal=causal, window=window, sinks=rng.choice([0, 1, 4, 70]) if window else 0)


# -------------------------------------------------------------------- inputs
def _lengths(case):
    """New tokens and keys of each sequence, from the case alone: ragged, the
    longest of them case["kv"] keys. Writing and attending sequences hold at
    least their new tokens."""
    R, kv, tokens = case["R"], case["kv"], case["tokens"]
    g = torch.Generator().manual_seed(1000003 * R + kv)
    new = [tokens // R + (1 if r < tokens % R else 0) for r in range(R)]
    part = torch.rand(R, generator=g).tolist()
    low = 0.25 if R > 1 else 1.0
    keys = [max(new[r], int(round(kv * (low + (1 - low) * part[r])))) for r in range(R)]
    keys[0] = max(new[0], kv)
    return new, keys


def _freqs(rot, scaled):
    """Inverse frequencies and the factor of cos and sin: plain, or blended
    between the plain and the 8 times slower ones by the turns a pair makes in
    the 4096 positions it was trained on."""
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "qk":
        B, N, hq, hkv, d = (case[x] for x in ("B", "N", "hq", "hkv", "d"))
        # the fused projection's output (B, N, heads, d), and views of it as (B, H, N, d)
        qkv = _randn((B, N, hq + 2 * hkv, d), gen)
        s["q"], s["k"], s["v"] = (x.transpose(1, 2) for x in qkv.split([hq, hkv, hkv], 2))
        start = torch.randint(0, max(1, case["far"] - N + 1), (B, 1), generator=gen, device="cuda")
        s["pos"] = (start + torch.arange(N, device="cuda")).to(torch.int32)
        f, s["rot_scale"] = _freqs(case["rot"], case["scaled"])
        s["freq"] = f.cuda()
        wt = F32 if case["wtype"] == "f32" else BF16
        s["wq"], s["wk"] = ((1 + 0.2 * _randn((d,), gen, F32)).to(wt) if case["norm"] else None for _ in range(2))
        if case["bwd"]:
            s["dq"], s["dk"], s["dv"] = (_randn((B, h, N, d), gen) for h in (hq, hkv, hkv))
        return s
    R, hkv, d, page = case["R"], case["hkv"], case["d"], case["page"]
    new, keys = _lengths(case)
    s["new"], s["keys"] = new, keys
    width = max(1, -(-max(keys) // page))
    n_pages = sum(-(-x // page) for x in keys) + 3
    # pages in an order of their own; places past a sequence's last page hold no page
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r in range(R):
        n = -(-keys[r] // page)
        table[r, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["q_off"] = torch.tensor([sum(new[:r]) for r in range(R + 1)], dtype=torch.int32, device="cuda")
    s["kv_off"] = torch.tensor([sum(keys[:r]) for r in range(R + 1)], dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(keys, dtype=torch.int32, device="cuda")
    for x in ("kc", "vc"):
        c = _randn((n_pages, hkv, page, d), gen)
        if case["e4m3"]:
            # rows of one scale each, as a write leaves them: largest value in (224, 448]
            top = c.abs().amax(-1, keepdim=True).to(F32)
            e = torch.ceil(torch.log2(top / 448.0))
            s[x] = (c.to(F32) * torch.exp2(-e)).to(E4M3)
            s[x + "_exp"] = (e.squeeze(-1) + 127).to(torch.uint8)
        else:
            s[x], s[x + "_exp"] = c, None
    if case["op"] == "write":
        s["k"], s["v"] = (_randn((case["tokens"], hkv, d), gen) for _ in range(2))
    if case["op"] == "attn":
        s["q"] = _randn((case["tokens"], case["hq"], d), gen)
        s["scale"] = d ** -0.5
    if own:
        # the handles a serving program keeps: checked views of the tensors above, nothing computed
        import mask_aware_sparse_gb300 as fm

        s["cache"] = fm.KVCache(s["kc"], s["vc"], s["kc_exp"], s["vc_exp"])
        s["batch"] = fm.PagedBatch(s["q_off"], s["kv_len"], s["table"])
    return s


# --------------------------------------------------------------- plain forms
def _angles(s):
    turn = s["pos"].to(F64)[..., None] * s["freq"].to(F64)  # far positions: 64 bits
    return (torch.cos(turn).to(F32) * s["rot_scale"])[:, None], (torch.sin(turn).to(F32) * s["rot_scale"])[:, None]


def _pairs(x, rot, inter):
    h = x[..., :rot]
    return (h[..., 0::2], h[..., 1::2]) if inter else (h[..., :rot // 2], h[..., rot // 2:])


def _unpair(a, b, rest, inter):
    h = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((h, rest), -1)


def _turn(x, cos, sin, rot, inter):
    a, b = _pairs(x, rot, inter)
    return _unpair(a * cos - b * sin, a * sin + b * cos, x[..., rot:], inter)


EPS = 1e-6


def _plain_qk(s):
    cos, sin = _angles(s)
    rot, inter = s["rot"], s["inter"]

    def forward(x, w):
        x = x.to(F32)
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(F32)
        return _turn(x, cos, sin, rot, inter).to(BF16).contiguous()

    def backward(dy, x, w):
        g = _turn(dy.to(F32), cos, -sin, rot, inter)
        if w is None:
            return g.to(BF16), None
        x = x.to(F32)
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        gw = g * w.to(F32)
        dx = r * gw - x * (r * r * r * (gw * x).mean(-1, keepdim=True))
        dw = (g * x * r).sum((0, 1, 2), dtype=F64)  # long sums: 64 bits
        return dx.to(BF16), dw.to(w.dtype)

    out = [forward(s["q"], s["wq"]), forward(s["k"], s["wk"]), s["v"].contiguous()]
    if s["bwd"]:
        (dq, dwq), (dk, dwk) = backward(s["dq"], s["q"], s["wq"]), backward(s["dk"], s["k"], s["wk"])
        # gradients in the projection's layout, as its own backward pass takes them
        lay = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
        out += [lay(dq), lay(dk), lay(s["dv"]), dwq, dwk]
    return out


def _plain_write(s):
    n = s["q_off"].long()
    t = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(n[1:].contiguous(), t, right=True)
    pos = s["kv_len"].long()[r] - (n[r + 1] - n[r]) + (t - n[r])
    page, slot = s["table"].long()[r, pos // s["page"]], pos % s["page"]
    out = []
    for x, c in ((s["k"], "kc"), (s["v"], "vc")):
        if s["e4m3"]:
            x = x.to(F32)
            top = x.abs().amax(-1, keepdim=True)
            m, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
            e = (e - 9 + (m > 0.875)).clamp(min=-126)
            e = torch.where(top > 0, e, torch.full_like(e, -126))
            s[c + "_exp"][page, :, slot] = (e.squeeze(-1) + 127).to(torch.uint8)
            s[c].view(torch.uint8)[page, :, slot] = torch.ldexp(x, -e).to(E4M3).view(torch.uint8)
            out += [s[c], s[c + "_exp"]]
        else:
            s[c][page, :, slot] = x
            out += [s[c]]
    return out


def _values(c, exp):
    return c.to(F32) if exp is None else c.to(F32) * torch.exp2(exp.to(F32) - 127)[..., None]


def _plain_read(s):
    n = s["kv_off"].long()
    i = torch.arange(sum(s["keys"]), device="cuda")
    r = torch.searchsorted(n[1:].contiguous(), i, right=True)
    j = i - n[r]
    page, slot = s["table"].long()[r, j // s["page"]], j % s["page"]
    out = []
    for c in ("kc", "vc"):
        exp = s[c + "_exp"]
        rows = _values(s[c][page, :, slot], None if exp is None else exp[page, :, slot])
        out.append(rows.to(BF16).transpose(0, 1).contiguous()[None])
    return out


def _plain_attn(s):
    R, page, hq, hkv, d = s["R"], s["page"], s["hq"], s["hkv"], s["d"]
    G, most, T = hq // hkv, max(s["new"]), s["tokens"]
    q_off, kv_len, table = s["q_off"].long(), s["kv_len"].long(), s["table"].long().clamp(min=0)
    # queries padded to (R, hkv, most * G, d), keys and values to (R, hkv, L, d)
    a = torch.arange(most, device="cuda")
    new = q_off[1:] - q_off[:-1]
    rows = (q_off[:-1, None] + a).clamp(max=T - 1)
    q = s["q"].to(F32)[rows].view(R, most, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, hkv, most * G, d)
    L = table.shape[1] * page
    take = lambda c, e: _values(c[table], None if e is None else e[table]).permute(0, 2, 1, 3, 4).reshape(R, hkv, L, d)  # noqa: E731
    j = torch.arange(L, device="cuda")
    held = (j < kv_len[:, None])[:, None, :, None]
    pos = (kv_len - new)[:, None] + a  # (R, most)
    see = (j < kv_len[:, None])[:, None, :] & torch.ones_like(pos, dtype=torch.bool)[:, :, None]
    if s["causal"]:
        see &= j <= pos[..., None]
    if s["window"]:
        see &= (j > pos[..., None] - s["window"]) | (j < s["sinks"])
    see = see.repeat_interleave(G, 1)[:, None]  # (R, 1, most * G, L)
    k = take(s["kc"], s["kc_exp"]).masked_fill(~held, 0.0)
    sc = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~see, -math.inf)
    del k
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = take(s["vc"], s["vc_exp"]).masked_fill(~held, 0.0)
    o = torch.matmul(p, v) / total.clamp(min=1e-30)
    lse = (top + torch.log(total)).squeeze(-1)
    there = (a < new[:, None]).nonzero(as_tuple=True)
    back = lambda x: x.view(R, hkv, most, G, -1).permute(0, 2, 1, 3, 4).reshape(R, most, hq, -1)[there]  # noqa: E731
    return [back(o).to(BF16), back(lse[..., None]).squeeze(-1)]


def run(state):
    s = state
    if not own:
        return {"qk": _plain_qk, "write": _plain_write, "read": _plain_read, "attn": _plain_attn}[s["op"]](s)
    import mask_aware_sparse_gb300 as fm

    if s["op"] == "qk":
        how = dict(positions=s["pos"], inv_freq=s["freq"], interleaved=s["inter"], rot_scale=s["rot_scale"],
                   q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
        out = list(fm.fm_qk_norm_rope(s["q"], s["k"], s["v"], **how))
        if s["bwd"]:
            out += list(fm.fm_qk_norm_rope_bwd(s["dq"], s["dk"], s["dv"], s["q"], s["k"], **how))
        return out
    if s["op"] == "write":
        fm.fm_cache_write(s["k"], s["v"], s["cache"], s["batch"])
        return [s[x] for x in ("kc", "kc_exp", "vc", "vc_exp") if s[x] is not None]
    if s["op"] == "read":
        return list(fm.fm_cache_read(s["cache"], s["kv_off"], s["table"], sum(s["keys"])))
    return list(fm.fm_attn_paged(s["q"], s["cache"], s["batch"], scale=s["scale"], causal=s["causal"],
                                 window=s["window"], sinks=s["sinks"]))


# ---------------------------------------------------------------------- work
def _seen(case):
    """(query, key) pairs, and keys that any query of their sequence sees."""
    new, keys = _lengths(case)
    pairs = cols = 0
    W, sinks = case["window"], case["sinks"]
    for n, L in zip(new, keys):
        if not case["causal"]:
            pairs, cols = pairs + n * L, cols + (L if n else 0)
            continue
        for p in range(L - n, L):
            pairs += p + 1 if not W else min(p + 1, W) + min(max(p + 1 - W, 0), sinks)
        if n:
            lo = max(0, L - n - W + 1) if W else 0
            cols += L - lo + min(lo, sinks)
    return pairs, cols


def work(case):
    if case["op"] == "qk":
        rows = case["B"] * case["N"]
        heads, d = case["hq"] + 2 * case["hkv"], case["d"]
        b = rows * heads * d * 4 + rows * 4
        if case["bwd"]:
            # dy read, dx written; with norms q and k are read again
            b += rows * heads * d * 4 + (rows * (case["hq"] + case["hkv"]) * d * 2 if case["norm"] else 0)
        return {"bytes": b, "flops": rows * heads * d * (20 if case["bwd"] else 8)}
    new, keys = _lengths(case)
    es = 1 if case["e4m3"] else 2
    row = case["hkv"] * (case["d"] * es + (1 if case["e4m3"] else 0))
    if case["op"] == "write":
        return {"bytes": 2 * case["tokens"] * (case["hkv"] * case["d"] * 2 + row), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * sum(keys) * (case["hkv"] * case["d"] * 2 + row), "flops": 0}
    pairs, cols = _seen(case)
    return {"bytes": 2 * cols * row + case["tokens"] * case["hq"] * (case["d"] * 4 + 4),
            "flops": 4 * pairs * case["hq"] * case["d"]}


# --------------------------------------------------------------------- exact
def _exact_qk(s):
    """The definition in 64 bits; gradients by differentiating it."""
    theta = s["pos"].double()[:, None, :, None] * s["freq"].double()
    z = torch.polar(torch.full_like(theta, s["rot_scale"]), theta)
    rot, inter = s["rot"], s["inter"]

    def f(x, w):
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
        head = x[..., :rot]
        if inter:
            c = torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous())
            head = torch.view_as_real(c * z).flatten(-2)
        else:
            c = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * z
            head = torch.cat((c.real, c.imag), -1)
        return torch.cat((head, x[..., rot:]), -1)

    out, grads, dws = [], [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x = x.detach().double().requires_grad_(s["bwd"])
        w = None if w is None else w.double().requires_grad_(s["bwd"])
        y = f(x, w)
        out.append(y.detach())
        if s["bwd"]:
            got = torch.autograd.grad(y, [x] if w is None else [x, w], dy.double())
            grads.append(got[0])
            dws.append(None if w is None else got[1])
    out.append(s["v"].double())
    return out + (grads + [s["dv"].double()] + dws if s["bwd"] else [])


def _exact_attn(s):
    """Sequence by sequence, keys gathered page by page, rows in blocks."""
    out = torch.zeros(s["tokens"], s["hq"], s["d"], dtype=F64, device="cuda")
    lse = torch.full((s["tokens"], s["hq"]), -math.inf, dtype=F64, device="cuda")
    G, at = s["hq"] // s["hkv"], 0
    for r, (n, L) in enumerate(zip(s["new"], s["keys"])):
        pages = s["table"][r, : -(-L // s["page"])].long()
        for h in range(s["hkv"] if n else 0):
            kv = []
            for c in ("kc", "vc"):
                x = s[c][pages, h].double()
                if s["e4m3"]:
                    x = x * torch.pow(2.0, s[c + "_exp"][pages, h].double() - 127)[..., None]
                kv.append(x.reshape(-1, s["d"])[:L])
            for a0 in range(0, n, 256):
                a1 = min(n, a0 + 256)
                q = s["q"][at + a0:at + a1, h * G:(h + 1) * G].double()
                w = torch.einsum("agd,jd->agj", q, kv[0]) * s["scale"]
                if s["causal"]:
                    away = torch.arange(L - n + a0, L - n + a1, device="cuda")[:, None] - torch.arange(L, device="cuda")
                    hide = away < 0
                    if s["window"]:
                        hide |= (away >= s["window"]) & (torch.arange(L, device="cuda") >= s["sinks"])
                    w = w.masked_fill(hide[:, None, :], -math.inf)
                lse[at + a0:at + a1, h * G:(h + 1) * G] = torch.logsumexp(w, -1)
                out[at + a0:at + a1, h * G:(h + 1) * G] = torch.einsum("agj,jd->agd", torch.softmax(w, -1), kv[1])
        at += n
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(s)
    if case["op"] == "attn":
        # 64-bit products at about a teraflop a second
        return _exact_attn(s) if work(case)["flops"] < 4e12 else None
    if case["op"] == "read":
        out = []
        for c in ("kc", "vc"):
            x = s[c].double()
            if s["e4m3"]:
                x = x * torch.pow(2.0, s[c + "_exp"].double() - 127)[..., None]
            rows = [x[s["table"][r, : -(-L // s["page"])].long()].transpose(0, 1).reshape(s["hkv"], -1, s["d"])[:, :L]
                    for r, L in enumerate(s["keys"])]
            out.append(torch.cat(rows, 1)[None])
        return out
    return None  # a write's rows are rounded to the cache's type by definition
