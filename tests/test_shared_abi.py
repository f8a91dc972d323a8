"""Appending with norm and rotation, page copies, attention over shared prefixes: what
the host side refuses, before any launch and without a GPU."""
import math

import pytest
import torch

import mask_aware_sparse_gb300 as fm
from test_serve_abi import A, ROWS, _batch, _cache, lib  # noqa: F401

I, U, W = fm.FM_ERR_INVALID_ARG, fm.FM_ERR_UNSUPPORTED, fm.FM_ERR_WORKSPACE
BAD_ROWS = (fm.fm_rows(A + 2, 128, 64), fm.fm_rows(A, 100, 64), fm.fm_rows(A, 128, 4), fm.fm_rows(0, 128, 64), None)


def _prob(**over):
    p = dict(B=1, N=3, H_q=4, H_kv=2, d=64, rot=32, interleaved=0, w_f32=1, eps=1e-6, rot_scale=1.0, pos=0, pos_sb=0,
             inv_freq=A, q_weight=A, k_weight=A)
    p.update(over)
    return fm.fm_qk_problem(*p.values())


def _groups(**over):
    s = dict(seq_off=A, prefix_len=A, S=1)
    s.update(over)
    return fm.fm_shared_prefix(*s.values())


@pytest.mark.parametrize("over, want", [
    (dict(k=0), I), (dict(v=A + 8), I), (dict(k_exp=A), I), (dict(n_pages=0), I), (dict(H_kv=0), I),
    (dict(page_size=8), U), (dict(d=96), U), (dict(n_pages=1 << 30, H_kv=4), U), (dict(n_pages=1, H_kv=65537), U),
])
def test_caches_refused(lib, over, want):  # noqa: F811
    c, b, s = _cache(**over), _batch(), _groups()
    assert lib.fm_cache_append(c, b, _prob(), ROWS, ROWS, ROWS, ROWS, 0) == want
    assert lib.fm_cache_copy(c, A, A, 3, 0) == want
    assert lib.fm_attn_shared(c, b, s, 3, 4, ROWS, 0.1, 1, ROWS, A, A, 1 << 30, 0) == want
    assert lib.fm_attn_shared_workspace_bytes(c, b, s, 3, 4) == 0


@pytest.mark.parametrize("over, T, want", [
    (dict(q_off=0), 3, I), (dict(kv_len=0), 3, I), (dict(page_table=0), 3, I), (dict(R=0), 3, I), (dict(width=0), 3, I),
    (dict(), -1, I), (dict(width=1 << 27), 3, U), (dict(), (1 << 30) + 1, U),
])
def test_batches_refused(lib, over, T, want):  # noqa: F811
    c, b = _cache(), _batch(**over)
    assert lib.fm_cache_append(c, b, _prob(N=T), ROWS, ROWS, ROWS, ROWS, 0) == want
    assert lib.fm_attn_shared(c, b, _groups(), T, 4, ROWS, 0.1, 1, ROWS, A, A, 1 << 30, 0) == want
    assert lib.fm_attn_shared_workspace_bytes(c, b, _groups(), T, 4) == 0


@pytest.mark.parametrize("over, want", [
    (dict(B=2), I), (dict(B=0), I), (dict(H_q=0), I), (dict(H_kv=1), I), (dict(d=128), I), (dict(d=96), U),
    (dict(rot=-16), I), (dict(rot=80), I), (dict(rot=24), U), (dict(eps=-1.0), I), (dict(eps=math.nan), I),
    (dict(rot_scale=math.inf), I), (dict(inv_freq=0), I), (dict(H_q=(1 << 20) + 1), U),
])
def test_append_arguments_refused(lib, over, want):  # noqa: F811
    assert lib.fm_cache_append(_cache(), _batch(), _prob(**over), ROWS, ROWS, ROWS, ROWS, 0) == want


def test_append_rows_refused(lib):  # noqa: F811
    c, b = _cache(), _batch()
    for bad in BAD_ROWS:
        for at in range(4):
            rows = [ROWS] * 4
            rows[at] = bad
            assert lib.fm_cache_append(c, b, _prob(), *rows, 0) == I
    assert lib.fm_cache_append(c, b, None, ROWS, ROWS, ROWS, ROWS, 0) == I
    assert lib.fm_cache_append(c, None, _prob(), ROWS, ROWS, ROWS, ROWS, 0) == I
    # nothing to do
    assert lib.fm_cache_append(c, b, _prob(N=0), None, None, None, None, 0) == fm.FM_OK


def test_copy_arguments_refused(lib):  # noqa: F811
    c = _cache()
    assert lib.fm_cache_copy(c, 0, A, 3, 0) == I and lib.fm_cache_copy(c, A, 0, 3, 0) == I
    assert lib.fm_cache_copy(c, A, A, -1, 0) == I and lib.fm_cache_copy(c, A, A, (1 << 30) + 1, 0) == U
    assert lib.fm_cache_copy(c, 0, 0, 0, 0) == fm.FM_OK


def test_shared_attention_arguments_refused(lib):  # noqa: F811
    c, b = _cache(), _batch()

    def call(s=_groups(), T=3, H_q=4, q=ROWS, scale=0.1, causal=1, o=ROWS, lse=A, ws=A, wsb=1 << 30):
        return lib.fm_attn_shared(c, b, s, T, H_q, q, scale, causal, o, lse, ws, wsb, 0)

    for bad in (None, _groups(seq_off=0), _groups(prefix_len=0), _groups(S=0), _groups(S=-2)):
        assert call(s=bad) == I
        assert lib.fm_attn_shared_workspace_bytes(c, b, bad, 3, 4) == 0
    assert call(s=_groups(S=1 << 30)) == U
    assert call(H_q=3) == I and call(H_q=0) == I and call(H_q=2 << 29) == U
    for s in (0.0, -1.0, math.nan, math.inf, 3.4e38):
        assert call(scale=s) == I
    for bad in BAD_ROWS:
        assert call(q=bad) == I and call(o=bad) == I
    assert call(lse=0) == I
    need = lib.fm_attn_shared_workspace_bytes(c, b, _groups(), 3, 4)
    assert need > 0
    assert call(ws=0) == W and call(wsb=need - 1) == W and call(ws=A + 8) == W
    assert call(T=0, q=None, o=None, lse=0, ws=0, wsb=0) == fm.FM_OK


def test_bindings_arguments_refused(lib, monkeypatch):  # noqa: F811
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    i32 = torch.int32
    for a in ((z(2, dt=i32), z(2, dt=i32)), (z(3, dt=i32), z(2, dt=torch.int64)), (z(1, dt=i32), z(0, dt=i32)),
              (z(3), z(2, dt=i32)), (z(3, 1, dt=i32), z(2, dt=i32)), (z(2, dt=i32), z(1, 1, dt=i32)),
              (z(3, dt=i32), z(2, dt=i32))):  # (the last: host tensors)
        with pytest.raises(ValueError):
            fm.SharedPrefix(*a)
    with pytest.raises(ValueError, match="KVCache"):
        fm.fm_cache_append(z(3, 4, 64), z(3, 2, 64), z(3, 2, 64), None, None)
    with pytest.raises(ValueError, match="KVCache"):
        fm.fm_cache_copy(None, z(3, dt=i32), z(3, dt=i32))
    with pytest.raises(ValueError, match="KVCache"):
        fm.fm_attn_shared(z(3, 4, 64), None, None, None, scale=0.1)
    # handles as they are after their checks, without a GPU
    cache, batch, groups = (object.__new__(t) for t in (fm.KVCache, fm.PagedBatch, fm.SharedPrefix))
    for name, x in dict(index=-1, H_kv=2, d=64, n_pages=1, page_size=16, k_exp=None, at=0, device="cpu").items():
        setattr(cache, name, x)
    for name, x in dict(index=-1, R=1, width=1, at=0).items():
        setattr(batch, name, x)
    for name, x in dict(index=-1, S=1, at=0).items():
        setattr(groups, name, x)
    monkeypatch.setattr(fm, "_enqueue", lambda *a: pytest.fail("reached the library"))
    monkeypatch.setattr(fm, "_shared_bytes", lambda *a: 1 << 10)
    q, k = z(3, 4, 64), z(3, 2, 64)
    f, pos = z(16, dt=torch.float32), z(3, dt=i32)
    for c in (dict(q=z(3, 4, 32)), dict(q=z(4, 64)), dict(q=q.float()), dict(k=z(2, 2, 64)), dict(v=z(3, 1, 64)),
              dict(q=z(3, 4, 128)[..., ::2]), dict(k=z(3, 2, 68)[..., 4:]), dict(inv_freq=f.double()),
              dict(inv_freq=z(1, 16, dt=torch.float32)), dict(positions=z(4, dt=i32)), dict(positions=pos.long()),
              dict(q_weight=z(32)), dict(q_weight=z(64), k_weight=z(64, dt=torch.float32)),
              dict(k_weight=z(64, dt=torch.float16)), dict(out=k), dict(out=q.float()), dict(out=q[:, :1].expand(3, 4, 64)),
              dict(q=z(3, 0, 64))):
        a = dict(q=q, k=k, v=k, positions=pos, inv_freq=f)
        a.update(c)
        with pytest.raises(ValueError):
            fm.fm_cache_append(a.pop("q"), a.pop("k"), a.pop("v"), cache, batch, **a)
    for src, dst in ((pos.long(), pos), (pos, pos[:2]), (pos[None], pos), (pos, z(3)), (z(6, dt=i32)[::2], pos)):
        with pytest.raises(ValueError):
            fm.fm_cache_copy(cache, src, dst)
    for c in (dict(q=z(3, 4, 32)), dict(q=z(3, 3, 64)), dict(q=z(3, 0, 64)), dict(q=q.float()), dict(shared=None),
              dict(o=k), dict(lse=z(3, 2, dt=torch.float32)), dict(lse=z(3, 4)), dict(ws=z(8, dt=torch.uint8)),
              dict(ws=z(1 << 10)), dict(o=q[:, :1].expand(3, 4, 64))):
        a = dict(q=q, shared=groups, scale=0.1)
        a.update(c)
        with pytest.raises(ValueError):
            fm.fm_attn_shared(a.pop("q"), cache, batch, a.pop("shared"), **a)
    groups.index = 1
    with pytest.raises(ValueError, match="another device"):
        fm.fm_attn_shared(q, cache, batch, groups, scale=0.1)
    # counts of which ctypes would keep the low 32 bits
    big = 2 ** 32 + 5
    groups.index = -1
    rows = z(1, 1, 64).expand(big, 2, 64)
    for call in (lambda: fm.fm_cache_append(rows, rows, rows, cache, batch),
                 lambda: fm.fm_attn_shared(rows, cache, batch, groups, scale=0.1),
                 lambda: fm.fm_cache_copy(cache, *[torch.empty(big, dtype=i32, device="meta")] * 2),
                 lambda: fm.SharedPrefix(torch.empty(big + 1, dtype=i32, device="meta"),
                                         torch.empty(big, dtype=i32, device="meta"))):
        with pytest.raises(ValueError, match="2\\^30"):
            call()


def test_bounds_of_prefixes(lib):  # noqa: F811
    # a program that leaves the bound as it finds it is not refused: below 0 it is not known, like 0
    c, b = _cache(), _batch()
    room = lib.fm_attn_shared_workspace_bytes(c, b, _groups(), 3, 4)
    for most in (-2 ** 31, -1, 0, 1, 2 ** 31 - 1):
        x = fm.fm_shared_prefix(A, A, 1, most)
        need = lib.fm_attn_shared_workspace_bytes(c, b, x, 3, 4)
        assert need > 0 and (most > 0 or need == room)
        assert lib.fm_attn_shared(c, b, x, 3, 4, ROWS, 0.1, 1, ROWS, A, A, need - 1, 0) == W
    off = torch.zeros(2, dtype=torch.int32)
    for most in (-1, 2 ** 30 + 1, 2 ** 32):
        with pytest.raises(ValueError, match="max_prefix"):
            fm.SharedPrefix(off, off[1:], max_prefix=most)
