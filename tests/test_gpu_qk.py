"""GPU: per-head norm and rotation of queries and keys, and its backward, against
the 64-bit formula, its differences, and inside flashmask_attention.

Bounds, per output element: one bf16 rounding (2^-8 relative) and the 32-bit
arithmetic before it: the norm's factor (sum of d products, a reciprocal root:
(d + 8) 2^-24), cos and sin (2^-22), four roundings of products and sums, all
relative to |a| + |b| of the rotated pair: below 2^-15 for d <= 256. Weight
gradients are sums of n terms |g x r| in 32 bits, each off by the same 2^-15,
added in chains of at most 2^12: below 2^-11 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import mask_aware_sparse_gb300 as fm
from serve_ref import BF16_HALF, qk_rows

pytestmark = pytest.mark.gpu
F32_REL = 2.0 ** -15


def _inputs(B, N, Hq, Hkv, d, seed, fused=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    return (q, k, v) if fused else tuple(t.contiguous() for t in (q, k, v))


def _close(got, want, mag, extra=0.0):
    got, want = got.detach().double().cpu(), want.detach()
    bound = BF16_HALF * want.abs() * 1.01 + (F32_REL + extra) * mag + 1e-30
    err = (got - want).abs()
    assert bool((err <= bound).all()), f"off by {float((err / bound).max()):.3g} of its bound"


def _mag(x, w, eps, rot, inter):
    """|a| + |b| of the pair an element belongs to, after the norm."""
    if w is not None:
        x = x * w.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    m = x.abs().clone()
    if rot:
        a = m[..., 0:rot:2] + m[..., 1:rot:2] if inter else m[..., :rot // 2] + m[..., rot // 2:rot]
        m[..., :rot] = torch.stack((a, a), -1).flatten(-2) if inter else torch.cat((a, a), -1)
    return m


CASES = [
    # B, N, Hq, Hkv, d, rot, interleaved, q norm, k norm, weights, positions from, shared positions
    (1, 1, 1, 1, 64, 64, False, True, True, torch.float32, 0, True),
    (2, 37, 6, 2, 64, 32, True, True, False, torch.bfloat16, 100000, False),
    (1, 130, 5, 1, 128, 128, False, True, True, torch.float32, -50, True),
    (3, 17, 4, 4, 128, 16, False, False, True, torch.bfloat16, 0, False),
    (1, 9, 32, 8, 128, 112, True, False, False, torch.float32, 2 ** 31 - 10, True),
    (2, 5, 3, 3, 256, 256, False, True, True, torch.float32, 1 << 20, False),
    (1, 70, 7, 1, 256, 48, True, True, True, torch.bfloat16, 7, True),
    (1, 4, 2, 2, 64, 0, False, True, True, torch.float32, 0, True),
    (1, 2600, 2, 1, 64, 64, True, True, True, torch.float32, 0, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("fused", [True, False])
def test_forward_and_backward(case, fused):
    B, N, Hq, Hkv, d, rot, inter, qn, kn, wt, start, shared = case
    q, k, v = _inputs(B, N, Hq, Hkv, d, 3, fused)
    g = torch.Generator().manual_seed(4)
    ws = [(1 + 0.3 * torch.randn(d, generator=g)).to(wt).cuda() if x else None for x in (qn, kn)]
    f, sc = fm.fm_rope_freqs(rot, kind="yarn", factor=4.0, orig_len=64, device="cuda") if rot else (None, 1.0)
    pos = (start + torch.arange(N, dtype=torch.int64))[None] - (0 if shared else torch.arange(B)[:, None] * 3)
    pos = pos.to(torch.int32)
    how = dict(positions=(pos[0] if shared else pos).cuda(), inv_freq=f, interleaved=inter, rot_scale=sc,
               q_weight=ws[0], k_weight=ws[1], eps=1e-5)
    out = fm.fm_qk_norm_rope(q, k, v, **how)
    grads = [torch.randn(t.shape, generator=g).to(torch.bfloat16).cuda() for t in (q, k, v)]
    back = fm.fm_qk_norm_rope_bwd(*grads, q, k, **how)
    again = fm.fm_qk_norm_rope_bwd(*grads, q, k, **how)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(back, again))  # sums in one order
    assert out[2].is_contiguous() and torch.equal(out[2], v) and torch.equal(back[2], grads[2])
    p2 = pos.expand(B, N)
    f64 = None if f is None else f.double().cpu()
    for i, (x, w) in enumerate(((q, ws[0]), (k, ws[1]))):
        x = x.detach().double().cpu().requires_grad_()
        w64 = None if w is None else w.detach().double().cpu().requires_grad_()
        y = qk_rows(x, w64, 1e-5, p2, f64, sc, inter)
        _close(out[i], y, sc * _mag(x, w64, 1e-5, rot, inter))
        dy = grads[i].double().cpu()
        want = torch.autograd.grad(y, [x] if w is None else [x, w64], dy)
        # |g w r| and |x r^3 mean(g w x)|, with |g| from the rotated pair
        gm = sc * _mag(dy, None, 0, rot, inter)
        if w is None:
            _close(back[i], want[0], gm)
            assert back[3 + i] is None
            continue
        xd = x.detach()
        r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + 1e-5)
        gw = gm * w64.detach().abs()
        _close(back[i], want[0], r * gw + xd.abs() * r ** 3 * (gw * xd.abs()).mean(-1, keepdim=True))
        dw = back[3 + i]
        assert dw.dtype == wt
        total = (gm * xd.abs() * r).sum((0, 1, 2))
        bound = 2.0 ** -11 * total + (BF16_HALF * want[1].abs() * 1.01 if wt == torch.bfloat16 else 0)
        assert bool(((dw.double().cpu() - want[1]).abs() <= bound).all())


def test_gradient_against_differences():
    # the function's own outputs are bf16, so differences are taken of the
    # 64-bit form at the kernel's gradient: <dx, t> = d/de <y(x + e t), dy>
    q, k, v = _inputs(1, 6, 2, 1, 64, 9)
    w = torch.linspace(0.5, 1.5, 64).cuda()
    f, _ = fm.fm_rope_freqs(64, device="cuda")
    pos = torch.arange(6, dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    dy, t = (torch.randn(q.shape, generator=g).to(torch.bfloat16) for _ in range(2))
    how = dict(positions=pos.cuda(), inv_freq=f, q_weight=w, eps=1e-6)
    dx = fm.fm_qk_norm_rope_bwd(dy.cuda(), k.contiguous(), None, q, k, **how)
    assert dx[2] is None and dx[4] is None
    x = q.double().cpu()
    y = lambda z: (qk_rows(z, w.cpu(), 1e-6, pos[None], f.cpu(), 1.0, False) * dy.double()).sum()  # noqa: E731
    e = 1e-4
    diff = float(y(x + e * t.double()) - y(x - e * t.double())) / (2 * e)
    got = float((dx[0].double().cpu() * t.double()).sum())
    # each element of dx is off by 2^-8 of itself (bf16); the difference by e^2
    bound = BF16_HALF * 1.1 * float((dx[0].double().cpu() * t.double()).abs().sum()) + 1e-4
    assert abs(diff - got) <= bound


def test_far_positions_are_exact():
    # 2^24 + 1 is no fp32 number: an fp32 product would turn by whole radians less
    pos = torch.tensor([2 ** 24 + 1, 2 ** 31 - 1, -(2 ** 31)], dtype=torch.int32)
    q = torch.ones(1, 1, 3, 64, dtype=torch.bfloat16).cuda()
    f = torch.ones(32, dtype=torch.float32) * 0.7
    out = fm.fm_qk_norm_rope(q, q.clone(), positions=pos.cuda(), inv_freq=f.cuda())
    want = qk_rows(q.double().cpu(), None, 0, pos[None], f, 1.0, False)
    _close(out[0], want, torch.full_like(want, 2.0))


def test_outputs_into_views_and_in_place():
    q, k, v = _inputs(2, 11, 4, 2, 128, 5)
    f, _ = fm.fm_rope_freqs(128, device="cuda")
    how = dict(positions=torch.arange(11, dtype=torch.int32).cuda(), inv_freq=f,
               q_weight=torch.ones(128).cuda(), k_weight=torch.ones(128).cuda())
    want = fm.fm_qk_norm_rope(q, k, v, **how)
    # token-major outputs, as the paged attention takes them
    tok = [torch.empty(2, 11, t.shape[1], 128, dtype=torch.bfloat16, device="cuda") for t in (q, k)]
    fm.fm_qk_norm_rope(q, k, out=tuple(t.transpose(1, 2) for t in tok), **how)
    for t, w in zip(tok, want):
        assert torch.equal(t.transpose(1, 2), w)
    fm.fm_qk_norm_rope(q, k, v, out=(q, k, v), **how)  # views of one projection, in place
    for t, w in zip((q, k, v), want):
        assert torch.equal(t, w)


def test_zero_and_non_finite_rows_stay_in_their_rows():
    q, k, v = _inputs(1, 8, 4, 2, 64, 6, fused=False)
    f, _ = fm.fm_rope_freqs(64, device="cuda")
    how = dict(positions=torch.arange(8, dtype=torch.int32).cuda(), inv_freq=f,
               q_weight=torch.ones(64).cuda(), k_weight=torch.ones(64).cuda())
    want = fm.fm_qk_norm_rope(q, k, **how)
    q2 = q.clone()
    q2[0, 1, 3] = float("nan")
    q2[0, 2, 4, 5] = float("inf")
    q2[0, 0, 0] = 0
    got = fm.fm_qk_norm_rope(q2, k, **how)
    assert torch.isnan(got[0][0, 1, 3]).all() and torch.isnan(got[0][0, 2, 4]).any()
    assert (got[0][0, 0, 0] == 0).all() and torch.equal(got[1], want[1])
    keep = torch.ones(4, 8, dtype=torch.bool)
    keep[1, 3] = keep[2, 4] = keep[0, 0] = False
    assert torch.equal(got[0][0][keep.cuda()], want[0][0][keep.cuda()])


@pytest.mark.parametrize("power", [-50, -20, 20, 50])
def test_rows_far_from_one(power):
    # squares stay in fp32's range, cubes of the norm's factor do not
    q, k, _ = _inputs(1, 5, 2, 2, 64, 7, fused=False)
    q, k = q * 2.0 ** power, k * 2.0 ** power
    w = torch.linspace(0.5, 1.5, 64).cuda()
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(q.shape, generator=g).to(torch.bfloat16)
    dq, dk, _, dwq, _ = fm.fm_qk_norm_rope_bwd(dy.cuda(), dy.cuda(), None, q, k, q_weight=w, k_weight=w, eps=0.0)
    for x, dx in ((q, dq), (k, dk)):
        x = x.double().cpu().requires_grad_()
        want = torch.autograd.grad(qk_rows(x, w.cpu(), 0.0, None, None, 1.0, False), x, dy.double())[0]
        xd, gw = x.detach(), dy.double().abs() * w.double().cpu()
        r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True))
        _close(dx, want, r * gw + xd.abs() * r ** 3 * (gw * xd.abs()).mean(-1, keepdim=True))


def test_captured_forward_and_backward():
    # a captured pass, replayed with other values beside an eager one on a second stream
    q, k, v = _inputs(2, 33, 4, 2, 128, 10)
    g = torch.Generator().manual_seed(5)
    grads = [torch.randn(t.shape, generator=g).to(torch.bfloat16).cuda() for t in (q, k, v)]
    f, _ = fm.fm_rope_freqs(128, device="cuda")
    w = torch.linspace(0.5, 1.5, 128).cuda()
    pos = torch.arange(33, dtype=torch.int32).cuda()
    how = dict(positions=pos, inv_freq=f, q_weight=w, k_weight=w)

    def step(stream=None):
        return (*fm.fm_qk_norm_rope(q, k, v, stream=stream, **how),
                *fm.fm_qk_norm_rope_bwd(*grads, q, k, stream=stream, **how))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    side = torch.cuda.Stream()
    for i in range(3):
        pos += 1000 * i
        q.copy_(torch.randn(q.shape, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        beside = step(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, beside))
    assert not torch.equal(held[0], q)


def test_flashmask_attention_with_norm_and_rotation():
    # the attention call's own path: same outputs and gradients as the steps
    # one by one, and as the differentiated 64-bit form within the parity bound
    import oracle
    from workloads import masks

    B, N, Hq, Hkv, d = 1, 300, 4, 2, 64
    q, k, v = _inputs(B, N, Hq, Hkv, d, 8)
    lens = [120, 100, 80]
    vec_np = [x[None] for x in masks.causal_documents(lens, N)]
    vec = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in vec_np]
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)  # packed documents restart
    f, sc = fm.fm_rope_freqs(d, device="cuda")
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    wq, wk = (torch.linspace(a, b, d).cuda().requires_grad_() for a, b in ((0.5, 1.5), (1.2, 0.8)))
    spec = fm.QKNormRope(positions=pos.cuda(), inv_freq=f, q_weight=wq, k_weight=wk)
    o = fm.flashmask_attention(*leaves, *vec, causal=True, qk=spec)
    g = torch.Generator().manual_seed(2)
    do = torch.randn(o.shape, generator=g).to(torch.bfloat16).cuda()
    o.backward(do)
    qn, kn, vn = fm.fm_qk_norm_rope(q, k, v, positions=pos.cuda(), inv_freq=f, q_weight=wq.detach(),
                                    k_weight=wk.detach())
    assert torch.equal(o, fm.flashmask_attention(qn, kn, vn, *vec, causal=True))
    f64 = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    O, _ = oracle.forward(f64(qn), f64(kn), f64(vn), vec_np, True, d ** -0.5)
    from helpers import GRAD_REL_L2, assert_out, rel_l2

    assert_out(f64(o), O)
    dQ, dK, dV = oracle.backward(f64(qn), f64(kn), f64(vn), f64(do), vec_np, True, d ** -0.5)
    for leaf, dn, w in ((leaves[0], dQ, wq), (leaves[1], dK, wk)):
        x = leaf.detach().double().cpu().requires_grad_()
        w64 = w.detach().double().cpu().requires_grad_()
        y = qk_rows(x, w64, 1e-6, pos[None], f.double().cpu(), 1.0, False)
        gx, gw = torch.autograd.grad(y, [x, w64], torch.from_numpy(dn))
        # the attention's gradients are within the parity bound, and one more bf16 rounding follows
        assert rel_l2(f64(leaf.grad), gx.numpy()) <= GRAD_REL_L2 + BF16_HALF
        assert rel_l2(f64(w.grad), gw.numpy()) <= GRAD_REL_L2 + BF16_HALF
    assert rel_l2(f64(leaves[2].grad), dV) <= GRAD_REL_L2
    assert fm.fm_device_status()[0] == fm.FM_OK
