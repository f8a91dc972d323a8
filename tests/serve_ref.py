"""Plain 64-bit forms of the norm and rotation, the paged cache and the
attention over it, written from their definitions (CPU, numpy / torch double),
with the bounds their kernels are held to."""
from __future__ import annotations

import math

import torch

BF16_HALF = 2.0 ** -8  # bf16: half a step, relative


def qk_rows(x, w, eps, pos, inv_freq, rot_scale, interleaved):
    """x (B, H, N, d) double -> normed and rotated, double. pos (B, N)."""
    if w is not None:
        x = x * w.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if inv_freq is None:
        return x
    th = pos.double()[:, None, :, None] * inv_freq.double()
    c, s = rot_scale * torch.cos(th), rot_scale * torch.sin(th)
    r = 2 * inv_freq.numel()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        head = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2:r]
        head = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((head, x[..., r:]), -1)


def quantised(x):
    """(value, exponent byte) of rows x (..., d) double as the cache keeps them."""
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(top)
    e = torch.ones_like(top)
    ok = ~bad & (top > 0)
    e[ok] = torch.ceil(torch.log2(top[ok] / 448.0)) + 127
    # log2's rounding: the smallest exponent that holds the row
    e = torch.where(ok & (top <= 448.0 * torch.exp2(e - 128)), e - 1, e)
    e = torch.where(ok & (top > 448.0 * torch.exp2(e - 127)), e + 1, e).clamp(1, 255)
    e[bad] = 255
    scale = torch.exp2(e - 127)[..., None]
    y = x / scale
    # e4m3: 4 significant bits, steps of 2^-9 below 2^-6, ties to even
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    v = torch.round(y / step) * step * scale
    v[bad] = math.nan
    return v, e.to(torch.uint8)


def paged(q, k, v, q_off, kv_len, scale, causal, window, sinks):
    """q (T, H, d), k / v: per sequence (H_kv, L, d), all double. Returns O, LSE,
    sum p |v| / l, and the largest scale * sum |q||k| of each row."""
    T, H, d = q.shape
    O, A = torch.zeros(T, H, d, dtype=torch.float64), torch.zeros(T, H, d, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    for r, L in enumerate(kv_len):
        t0, n = q_off[r], q_off[r + 1] - q_off[r]
        if n == 0:
            continue
        G = H // k[r].shape[0]
        kk, vv = (x.repeat_interleave(G, 0) for x in (k[r], v[r]))  # (H, L, d)
        qq = q[t0:t0 + n].transpose(0, 1)
        s = qq @ kk.transpose(1, 2) * scale
        p = (L - n + torch.arange(n))[:, None]
        j = torch.arange(L)
        see = torch.ones(n, L, dtype=torch.bool)
        if causal:
            see = j <= p
            if window:
                see = see & ((j > p - window) | (j < sinks))
        s = s.masked_fill(~see, -math.inf)
        some = see.any(-1)
        z = torch.logsumexp(s, -1)
        w = torch.where(some[None, :, None], torch.exp(s - z[..., None].nan_to_num(neginf=0.0)), torch.zeros_like(s))
        O[t0:t0 + n] = (w @ vv).transpose(0, 1)
        A[t0:t0 + n] = (w @ vv.abs()).transpose(0, 1)
        lse[t0:t0 + n] = z.transpose(0, 1)
        if L:
            mag[t0:t0 + n] = (qq.abs() @ kk.abs().transpose(1, 2)).amax(-1).transpose(0, 1) * scale
    return O, lse, A, mag


def assert_paged(o, lse, ref, d):
    """O and LSE against `paged`. A score is a sum of d products in 32 bits: off by
    at most (d + 2) 2^-24 scale sum |q||k| <= ds, its exponential by ds + 2^-21
    relative; p is rounded to bf16 at most once (2^-8 relative), O once."""
    O, L, A, mag = ref
    ds = (d + 2) * 2.0 ** -24 * mag + 2.0 ** -21
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(L)), "rows without keys differ"
    bound = (BF16_HALF + 2 * ds[..., None]) * A * 1.02 + BF16_HALF * O.abs() * 1.02 + 1e-30
    err = (o - O).abs()
    assert bool((err <= bound).all()), f"O off by {float((err / bound).max()):.3g} of its bound"
    ok = ~torch.isneginf(L)
    if ok.any():
        lb = 2 * ds[ok] + L[ok].abs() * 2.0 ** -22 + 2.0 ** -20
        le = (lse[ok] - L[ok]).abs()
        assert bool((le <= lb).all()), f"LSE off by {float((le / lb).max()):.3g} of its bound"
