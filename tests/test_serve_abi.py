"""Norm and rotation, paged cache and attention over it: what the host side
refuses, before any launch and without a GPU, and the host functions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import mask_aware_sparse_gb300 as fm
from mask_aware_sparse_gb300 import build as fmbuild

A = 1 << 20  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    fmbuild.build()
    return fm.lib()


def _cache(**over):
    c = dict(k=A, v=A, k_exp=0, v_exp=0, n_pages=4, H_kv=2, page_size=16, d=64)
    c.update(over)
    return fm.fm_kv_cache(*c.values())


def _batch(**over):
    b = dict(q_off=A, kv_len=A, page_table=A, R=2, width=3)
    b.update(over)
    return fm.fm_paged_batch(*b.values())


ROWS = fm.fm_rows(A, 128, 64)


@pytest.mark.parametrize("over, want", [
    (dict(k=0), "INVALID_ARG"), (dict(v=A + 8), "INVALID_ARG"), (dict(k_exp=A), "INVALID_ARG"),
    (dict(k_exp=A + 4, v_exp=A), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"), (dict(H_kv=0), "INVALID_ARG"),
    (dict(n_pages=-1), "INVALID_ARG"), (dict(page_size=8), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"),
    (dict(page_size=256), "UNSUPPORTED"), (dict(d=96), "UNSUPPORTED"), (dict(d=0), "UNSUPPORTED"),
    (dict(n_pages=1 << 30, H_kv=4), "UNSUPPORTED"), (dict(n_pages=1, H_kv=65537), "UNSUPPORTED"),
])
def test_caches_refused(lib, over, want):
    want = getattr(fm, "FM_ERR_" + want)
    c, b = _cache(**over), _batch()
    assert lib.fm_cache_write(c, b, 3, ROWS, ROWS, 0) == want
    assert lib.fm_cache_read(c, A, A, 2, 3, 5, A, A, 0) == want
    assert lib.fm_attn_paged(c, b, 3, 4, ROWS, 0.1, 1, 0, 0, ROWS, A, A, 1 << 30, 0) == want
    assert lib.fm_attn_paged_workspace_bytes(c, b, 3, 4) == 0


@pytest.mark.parametrize("over, T, want", [
    (dict(q_off=0), 3, "INVALID_ARG"), (dict(kv_len=0), 3, "INVALID_ARG"), (dict(page_table=0), 3, "INVALID_ARG"),
    (dict(R=0), 3, "INVALID_ARG"), (dict(width=0), 3, "INVALID_ARG"), (dict(width=-2), 3, "INVALID_ARG"),
    (dict(), -1, "INVALID_ARG"), (dict(width=1 << 27), 3, "UNSUPPORTED"), (dict(), (1 << 30) + 1, "UNSUPPORTED"),
])
def test_batches_refused(lib, over, T, want):
    want = getattr(fm, "FM_ERR_" + want)
    c, b = _cache(), _batch(**over)
    assert lib.fm_cache_write(c, b, T, ROWS, ROWS, 0) == want
    assert lib.fm_attn_paged(c, b, T, 4, ROWS, 0.1, 1, 0, 0, ROWS, A, A, 1 << 30, 0) == want


def test_attention_arguments_refused(lib):
    c, b, I = _cache(), _batch(), fm.FM_ERR_INVALID_ARG

    def call(T=3, H_q=4, q=ROWS, scale=0.1, causal=1, window=0, sinks=0, o=ROWS, lse=A, ws=A, wsb=1 << 30):
        return lib.fm_attn_paged(c, b, T, H_q, q, scale, causal, window, sinks, o, lse, ws, wsb, 0)

    assert call(H_q=3) == I and call(H_q=0) == I
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=s) == I
    assert call(window=-1) == I and call(window=4, sinks=-1) == I
    assert call(causal=0, window=4) == I and call(causal=0, sinks=1) == I
    assert call(q=None) == I and call(o=None) == I and call(lse=0) == I
    for bad in (fm.fm_rows(A + 2, 128, 64), fm.fm_rows(A, 100, 64), fm.fm_rows(A, 128, 4), fm.fm_rows(0, 128, 64)):
        assert call(q=bad) == I and call(o=bad) == I
        assert lib.fm_cache_write(c, b, 3, bad, ROWS, 0) == I and lib.fm_cache_write(c, b, 3, ROWS, bad, 0) == I
    need = lib.fm_attn_paged_workspace_bytes(c, b, 3, 4)
    assert need > 0
    assert call(ws=0) == fm.FM_ERR_WORKSPACE and call(wsb=need - 1) == fm.FM_ERR_WORKSPACE
    assert call(ws=A + 8) == fm.FM_ERR_WORKSPACE
    assert call(H_q=2 << 29) == fm.FM_ERR_UNSUPPORTED
    # nothing to do
    assert call(T=0, q=None, o=None, lse=0, ws=0, wsb=0) == fm.FM_OK
    assert lib.fm_cache_write(c, b, 0, None, None, 0) == fm.FM_OK
    assert lib.fm_cache_read(c, A, A, 2, 3, 0, 0, 0, 0) == fm.FM_OK
    assert lib.fm_cache_read(c, 0, A, 2, 3, 5, A, A, 0) == I
    assert lib.fm_cache_read(c, A, A, 2, 3, -5, A, A, 0) == I
    assert lib.fm_cache_read(c, A, A, 2, 3, 5, A + 2, A, 0) == I


def test_norm_rotation_arguments_refused(lib):
    I, U = fm.FM_ERR_INVALID_ARG, fm.FM_ERR_UNSUPPORTED
    V = fm.fm_view(A, 1024, 64, 128)

    def prob(**over):
        p = dict(B=1, N=4, H_q=2, H_kv=1, d=64, rot=32, interleaved=0, w_f32=1, eps=1e-6, rot_scale=1.0, pos=A,
                 pos_sb=0, inv_freq=A, q_weight=A, k_weight=A)
        p.update(over)
        return fm.fm_qk_problem(*p.values())

    def fwd(p, q=V, k=V, v=V, qo=V, ko=V, vo=V):
        return lib.fm_qk_norm_rope(p, q, k, v, qo, ko, vo, 0)

    def bwd(p, g=(V, V, V), x=(V, V), d=(V, V, V), dwq=A, dwk=A, ws=A, wsb=1 << 30):
        return lib.fm_qk_norm_rope_bwd(p, *g, *x, *d, dwq, dwk, ws, wsb, 0)

    for over, want in ((dict(B=-1), I), (dict(N=-1), I), (dict(H_q=0), I), (dict(H_kv=0), I), (dict(d=96), U),
                       (dict(rot=-16), I), (dict(rot=80), I), (dict(rot=24), U), (dict(eps=-1.0), I),
                       (dict(eps=math.nan), I), (dict(eps=math.inf), I), (dict(rot_scale=math.nan), I),
                       (dict(pos=0), I), (dict(inv_freq=0), I), (dict(B=1 << 16, N=1 << 16), U)):
        assert fwd(prob(**over)) == want, over
        assert bwd(prob(**over)) == want, over
    assert lib.fm_qk_norm_rope(None, V, V, V, V, V, V, 0) == I
    for bad in (None, fm.fm_view(0, 0, 0, 0), fm.fm_view(A + 8, 0, 0, 0), fm.fm_view(A, 4, 0, 0),
                fm.fm_view(A, 0, 2, 0), fm.fm_view(A, 0, 0, 1)):
        for where in ("q", "k", "v", "qo", "ko", "vo"):
            assert fwd(prob(), **{where: bad}) == I, where
        for i in range(3):
            g = [V, V, V]
            g[i] = bad
            assert bwd(prob(), g=g) == I and bwd(prob(), d=g) == I
        assert bwd(prob(), x=(bad, V)) == I and bwd(prob(), x=(V, bad)) == I
    assert bwd(prob(), dwq=0) == I and bwd(prob(), dwk=0) == I
    need = lib.fm_qk_norm_rope_bwd_workspace_bytes(prob())
    assert need > 0 and lib.fm_qk_norm_rope_bwd_workspace_bytes(prob(q_weight=0, k_weight=0)) == 0
    assert bwd(prob(), ws=A + 4) == fm.FM_ERR_WORKSPACE
    assert bwd(prob(), ws=0) == fm.FM_ERR_WORKSPACE and bwd(prob(), wsb=need - 1) == fm.FM_ERR_WORKSPACE
    assert fwd(prob(B=0), q=None, k=None) == fm.FM_OK and fwd(prob(N=0)) == fm.FM_OK
    assert bwd(prob(B=0, q_weight=0, k_weight=0)) == fm.FM_OK


def test_rope_freqs(lib):
    rot, base = 64, 10000.0
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    close = lambda t, x: np.testing.assert_allclose(t.numpy(), x.astype(np.float32), rtol=2 ** -23)  # noqa: E731
    f, s = fm.fm_rope_freqs(rot, base=base)
    close(f, plain)
    assert s == 1.0
    f, s = fm.fm_rope_freqs(rot, base=base, kind="linear", factor=4.0)
    close(f, plain / 4)
    assert s == 1.0
    f, s = fm.fm_rope_freqs(rot, base=base, kind="ntk", factor=4.0)
    close(f, (base * 4.0 ** (rot / (rot - 2))) ** (-2.0 * i / rot))
    assert s == 1.0 and f[0] == 1.0
    # the slowest pair of the NTK base turns as slowly as the interpolated one
    np.testing.assert_allclose(float(f[-1]), plain[-1] / 4, rtol=1e-6)
    f, s = fm.fm_rope_freqs(rot, base=base, kind="yarn", factor=8.0, orig_len=4096)
    turns = 4096 * plain / (2 * math.pi)
    y = f.numpy()
    np.testing.assert_allclose(s, 0.1 * math.log(8.0) + 1.0, rtol=1e-6)
    # kept where a pair turns much more than 32 times, interpolated below one turn, in between otherwise
    assert np.allclose(y[turns > 48], plain[turns > 48], rtol=1e-6)
    assert np.allclose(y[turns < 0.7], plain[turns < 0.7] / 8, rtol=1e-6)
    assert ((y <= plain * (1 + 1e-6)) & (y >= plain / 8 * (1 - 1e-6))).all() and (np.diff(y) < 0).all()
    for bad in (dict(rot=0), dict(rot=3), dict(base=1.0), dict(base=math.inf), dict(factor=0.5), dict(factor=math.nan),
                dict(kind="ntk", rot=2), dict(kind="yarn"), dict(kind="yarn", orig_len=8, beta_fast=1.0, beta_slow=2.0),
                dict(kind="yarn", orig_len=8, beta_slow=0.0)):
        with pytest.raises(fm.FMError):
            fm.fm_rope_freqs(**{"rot": 64, **bad})
    with pytest.raises(ValueError):
        fm.fm_rope_freqs(64, kind="other")


def test_binding_checks_before_any_library_call(lib):
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731
    kc = z(4, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fm.KVCache(kc, kc.clone())
    for k, v, e in ((z(4, 2, 16), kc, ()), (kc, z(4, 2, 32, 64), ()), (kc.float(), kc, ()),
                    (z(4, 2, 8, 64), z(4, 2, 8, 64), ()), (z(4, 2, 16, 80), z(4, 2, 16, 80), ()),
                    (kc, kc, (z(4, 2, 16, dt=torch.uint8),)),
                    (kc.to(torch.float8_e4m3fn), kc.to(torch.float8_e4m3fn), (z(4, 2, 8, dt=torch.uint8),) * 2),
                    (kc.to(torch.float8_e4m3fn), kc.to(torch.float8_e4m3fn), ()),
                    (kc.transpose(0, 1), kc.transpose(0, 1), ())):
        with pytest.raises(ValueError):
            fm.KVCache(k, v, *e)
    for a in ((z(3, dt=i32), z(2, dt=i32), z(2, dt=i32)), (z(2, dt=i32), z(2, dt=i32), z(2, 3, dt=i32)),
              (z(3, dt=i32), z(3, dt=i32), z(2, 3, dt=i32)), (z(3, dt=i32), z(2, dt=i32), z(2, 3, dt=torch.int64)),
              (z(3, dt=i32), z(2, dt=i32), z(2, 0, dt=i32)), (z(3, dt=i32), z(2, dt=i32), z(2, 3, dt=i32))):
        with pytest.raises(ValueError):
            fm.PagedBatch(*a)
    with pytest.raises(ValueError):
        fm.fm_cache_new(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="KVCache"):
        fm.fm_attn_paged(z(3, 4, 64), None, None, scale=0.1)
    with pytest.raises(ValueError, match="KVCache"):
        fm.fm_cache_write(z(3, 2, 64), z(3, 2, 64), None, None)
    q, k = z(1, 4, 8, 64), z(1, 2, 8, 64)
    f, pos = z(16, dt=torch.float32), z(8, dt=i32)
    cases = [dict(k=z(1, 2, 9, 64)), dict(k=z(2, 8, 64)), dict(v=z(1, 2, 8, 32)), dict(positions=z(9, dt=i32)),
             dict(positions=pos.long()), dict(positions=None), dict(inv_freq=f.double()), dict(q_weight=z(32)),
             dict(q_weight=z(64), k_weight=z(64, dt=torch.float32)), dict(q_weight=z(64, dt=torch.float16)),
             dict(q=z(1, 4, 8, 128)[..., ::2]), dict(q=z(1, 4, 8, 68)[..., 4:]), dict(q=q.float()),
             dict(out=(q,)), dict(out=(q, q, k)), dict(out=(q[:, :1].expand(1, 4, 8, 64), k, k))]
    for c in cases:
        a = dict(q=q, k=k, v=k, positions=pos, inv_freq=f)
        a.update(c)
        with pytest.raises(ValueError):
            fm.fm_qk_norm_rope(a.pop("q"), a.pop("k"), a.pop("v"), **a)
    with pytest.raises(ValueError, match="CUDA"):
        fm.fm_qk_norm_rope(q, k, k, positions=pos, inv_freq=f)
    with pytest.raises(ValueError, match="CUDA"):
        fm.fm_qk_norm_rope_bwd(q, k, k, q, k, positions=pos, inv_freq=f)
    with pytest.raises(ValueError, match="shape"):
        fm.fm_qk_norm_rope_bwd(k, k, k, q, k, positions=pos, inv_freq=f)


def test_second_derivatives_are_refused(monkeypatch):
    # the library's calls stand for themselves here: what matters is that a gradient's own
    # gradient raises, where it used to leave the calls' part out
    x = torch.randn(3, 1, 2, 4, 64, dtype=torch.float64)
    monkeypatch.setattr(fm, "fm_qk_norm_rope", lambda q, k, v, **kw: (2 * q, 3 * k, v.clone()))
    monkeypatch.setattr(fm, "fm_qk_norm_rope_bwd", lambda a, b, c, q, k, **kw: (2 * a * q, 3 * b, c, None, None))
    monkeypatch.setattr(fm, "attn_tiling", lambda: (128, 128))
    monkeypatch.setattr(fm, "fm_classify_tiles", lambda *a, **kw: None)
    monkeypatch.setattr(fm, "fm_attn_fwd", lambda q, k, v, *a, **kw: (q * k * v, None))
    monkeypatch.setattr(fm, "fm_attn_bwd", lambda q, k, v, o, lse, do, *a, **kw: (do * k * v, do * q * v, do * q * k))
    for spec in (None, fm.QKNormRope()):
        for of in (lambda o: o.sum(), lambda o: (o * o).sum()):
            q, k, v = (t.clone().requires_grad_() for t in x)
            o = fm.flashmask_attention(q, k, v, None, None, None, None, causal=True, qk=spec)
            first = torch.autograd.grad(of(o), (q, k, v), create_graph=True)
            assert all(g.abs().sum() > 0 for g in first)
            for again in (lambda: torch.autograd.grad(sum(g.sum() for g in first), (q, k, v)),
                          lambda: (of(o) + sum((g * g).sum() for g in first)).backward()):
                with pytest.raises(RuntimeError, match="second derivatives"):
                    again()
            # the gradients by themselves are as without create_graph: tensors of their own, no views
            assert not any(g._is_view() for g in first)
            o = fm.flashmask_attention(q, k, v, None, None, None, None, causal=True, qk=spec)
            for a, b in zip(first, torch.autograd.grad(of(o), (q, k, v))):
                assert torch.equal(a, b) and not b.requires_grad


def test_a_stream_of_another_device_is_refused(monkeypatch):
    # torch's and the library's calls stand for themselves: two devices, the first one current
    import contextlib

    at = [0]

    @contextlib.contextmanager
    def on(dev):
        was, at[0] = at[0], dev
        yield
        at[0] = was

    ran = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "stream", on)  # a stream is its device's index here
    monkeypatch.setattr(fm, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(fm, "_fast_fn", lambda name: lambda *a: ran.append((at[0], a)) or fm.FM_OK)
    call = fm._streamed(lambda dev: fm._enqueue("fm_cache_write", dev, 7))
    call(0)
    call(1)  # the tensors' device, its current stream
    call(1, stream=1)
    assert ran == [(0, (7, 100)), (1, (7, 101)), (1, (7, 101))]
    for dev, stream in ((0, 1), (1, 0)):
        if stream == 0:
            at[0] = 1
        with pytest.raises(ValueError, match="another device"):
            call(dev, stream=stream)
    at[0] = 0
    call(1)  # a refused call leaves nothing behind
    assert len(ran) == 4


@pytest.mark.parametrize("rot, base, orig_len", [(64, 10000.0, 1), (64, 10000.0, 6), (16, 500000.0, 5),
                                                 (64, 10000.0, 2 ** 40), (32, 1.5, 10 ** 6)])
def test_yarn_where_all_pairs_are_slow_or_fast(lib, rot, base, orig_len):
    # every pair turns less than once, or more than 32 times, within the trained length
    plain = base ** (-2.0 * np.arange(rot // 2) / rot)
    turns = orig_len * plain / (2 * math.pi)
    assert (turns < 1).all() or (turns > 32).all()
    f, _ = fm.fm_rope_freqs(rot, base=base, kind="yarn", factor=8.0, orig_len=orig_len)
    np.testing.assert_allclose(f.numpy(), plain / (8.0 if turns[0] < 1 else 1.0), rtol=2 ** -23)


@pytest.mark.parametrize("scale, want", [(2.0 ** 127, "WORKSPACE"), (2.5e38, "INVALID_ARG"), (3.4e38, "INVALID_ARG"),
                                         (1e-45, "WORKSPACE")])
def test_scales_that_leave_fp32_in_log2_units_refused(lib, scale, want):
    assert lib.fm_attn_paged(_cache(), _batch(), 3, 4, ROWS, scale, 1, 0, 0, ROWS, A, 0, 0, 0) == getattr(fm, "FM_ERR_" + want)


def test_counts_beyond_32_bits_refused_by_the_binding(lib, monkeypatch):
    # ctypes keeps the low 32 bits of a larger number: 2^32 + 5 tokens would be five
    i32, big = torch.int32, 2 ** 32 + 5
    on_meta = lambda *s, dt=i32: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    for R, width in ((1, big), (big, 1)):
        with pytest.raises(ValueError, match="2\\^30"):
            fm.PagedBatch(on_meta(R + 1), on_meta(R), on_meta(R, width))
    # handles as they are after their checks, without a GPU
    cache, batch = object.__new__(fm.KVCache), object.__new__(fm.PagedBatch)
    for name, x in dict(index=-1, H_kv=1, d=64, n_pages=1, page_size=16, k_exp=None, at=0, device="cpu").items():
        setattr(cache, name, x)
    for name, x in dict(index=-1, R=1, width=1, at=0).items():
        setattr(batch, name, x)
    rows = torch.zeros(1, 1, 64, dtype=torch.bfloat16).expand(big, 1, 64)
    monkeypatch.setattr(fm, "_enqueue", lambda *a: pytest.fail("reached the library"))
    monkeypatch.setattr(fm, "_paged_bytes", lambda *a: pytest.fail("reached the library"))
    with pytest.raises(ValueError, match="2\\^30"):
        fm.fm_cache_write(rows, rows, cache, batch)
    with pytest.raises(ValueError, match="2\\^30"):
        fm.fm_attn_paged(rows, cache, batch, scale=0.1)
    for T, H in ((big, 1), (-1, 1), (1, big), (1, 0)):
        with pytest.raises(ValueError, match="2\\^30"):
            fm.fm_attn_paged_workspace_bytes(cache, batch, T, H)


@pytest.mark.parametrize("how", [dict(rot=2 ** 32 + 64), dict(rot=64, kind="yarn", factor=2.0, orig_len=2 ** 64 + 4096)])
def test_rotations_beyond_the_librarys_integers_refused(lib, how):
    with pytest.raises(ValueError, match="too large"):
        fm.fm_rope_freqs(**how)
