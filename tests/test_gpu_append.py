"""GPU: new tokens appended to the paged cache with norm and rotation, and pages copied
to pages.

Queries, values and the keys of a bf16 cache are held to the bits of the two calls that
the append stands for. Keys of an e4m3 cache are rounded once, from 32 bits: a key is
within 2^-15 of its pair's magnitudes before that (test_gpu_qk derives it), its stored
value within half a step of e4m3: 2^-4 of it, or 2^-10 of the scale where its steps are
absolute; the scale is the smallest that holds the row's largest magnitude, which is
known within the same 2^-15."""
import pytest
import torch

import mask_aware_sparse_gb300 as fm
from serve_ref import qk_rows, quantised
from test_gpu_paged import Setup
from test_gpu_qk import F32_REL, _mag

pytestmark = pytest.mark.gpu
RANGE = (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE)
OK = (fm.FM_OK, 0)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _state(cache):
    return [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp) if t is not None]


CASES = [
    # new, keys, Hq, Hkv, d, page, rot, interleaved, q norm, k norm, weights, positions given
    ([1], [1], 1, 1, 64, 16, 64, False, True, True, torch.float32, False),
    ([1, 1, 1], [40, 17, 90], 32, 8, 128, 16, 128, False, True, True, torch.bfloat16, False),
    ([5, 0, 37], [9, 30, 37], 6, 2, 64, 32, 32, True, True, False, torch.bfloat16, True),
    ([130], [200], 5, 1, 128, 64, 128, True, False, True, torch.float32, False),
    ([17, 3], [17, 300], 3, 3, 256, 128, 48, False, True, True, torch.float32, True),
    ([700, 2], [1500, 2], 7, 1, 256, 16, 256, True, True, True, torch.float32, False),
    ([9, 4], [60, 4], 2, 2, 64, 16, 0, False, True, True, torch.float32, False),
    ([2600], [2600], 2, 1, 64, 64, 64, False, False, False, torch.float32, False),
    ([3000, 1, 1111], [3000, 700, 1200], 16, 4, 128, 64, 112, False, True, True, torch.bfloat16, False),
    ([1] * 300, [20] * 300, 4, 3, 64, 32, 16, False, True, True, torch.float32, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}-{sum(c[0])}-" + "-".join(str(x).replace("torch.", "") for x in c[2:]))
@pytest.mark.parametrize("f8", [False, True])
def test_append_is_norm_rotation_and_write(case, f8):
    new, keys, Hq, Hkv, d, page, rot, inter, qn, kn, wdt, given = case
    s = Setup(keys, new, Hkv, d, page, f8, seed=60)
    T = sum(new)
    qkv = torch.randn(T + 2, Hq + 2 * Hkv, d, generator=s.g).to(torch.bfloat16).cuda()  # two tokens of no sequence
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    f, sc = fm.fm_rope_freqs(rot, kind="yarn", factor=4.0, orig_len=64, device="cuda") if rot else (None, 1.0)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=s.g)).to(wdt).cuda() if n else None for n in (qn, kn))
    place = torch.cat([torch.arange(L - n, L) for n, L in zip(new, keys)] + [torch.zeros(2)]).int()
    pos = torch.randint(-100, 1 << 20, (T + 2,), generator=s.g).int() if given else place
    how = dict(inv_freq=f, interleaved=inter, rot_scale=sc, q_weight=wq, k_weight=wk, eps=1e-5)
    before = _state(s.cache)
    out = torch.full((T + 2, Hq + 1, d), 7.0, dtype=torch.bfloat16).cuda()
    got = fm.fm_cache_append(q, k, v, s.cache, s.batch, positions=pos.cuda() if given else None, out=out[:, 1:], **how)
    assert fm.fm_device_status() == OK
    assert got.data_ptr() == out[:, 1:].data_ptr() and (out[:, 0] == 7).all() and (out[T:] == 7).all()
    state = _state(s.cache)
    # the two calls, from the same cache
    for t, b in zip((t for t in (s.cache.k, s.cache.v, s.cache.k_exp, s.cache.v_exp) if t is not None), before):
        t.view(torch.uint8).copy_(b)
    view = lambda t: t[:T].transpose(0, 1)[None]  # noqa: E731
    qr, kr = fm.fm_qk_norm_rope(view(q), view(k), positions=pos[:T].cuda() if rot else None, **how)
    assert torch.equal(qr[0].transpose(0, 1), out[:T, 1:])
    fm.fm_cache_write(kr[0].transpose(0, 1), v[:T], s.cache, s.batch)
    want = _state(s.cache)
    if not f8:
        assert all(torch.equal(a, b) for a, b in zip(state, want))
        return
    assert torch.equal(state[1], want[1]) and torch.equal(state[3], want[3])
    # keys: places that the write does not touch are untouched
    seq = torch.cat([torch.full((n,), r) for r, n in enumerate(new)]).long()
    pg = s.table.cpu()[seq, place[:T].long() // page].long()
    slot = place[:T].long() % page
    hit = torch.zeros(s.cache.k.shape[0], page, dtype=torch.bool)
    hit[pg, slot] = True
    hit = hit[:, None].expand(-1, Hkv, -1)
    for i in (0, 2):
        assert torch.equal(state[i].cpu()[~hit], before[i].cpu()[~hit])
    # those that it does hold the rotated keys
    x = k[:T].double().cpu().transpose(0, 1)[None]
    ref = qk_rows(x, None if wk is None else wk.cpu(), 1e-5, pos[None, :T], None if f is None else f.cpu(), sc, inter)
    mag = _mag(x, None if wk is None else wk.cpu(), 1e-5, rot, inter) * max(1.0, sc)
    ref, off = (t[0].transpose(0, 1) for t in (ref, F32_REL * mag))  # (T, Hkv, d)
    stored = state[0].cpu()[pg, :, slot].contiguous().view(torch.float8_e4m3fn).double()
    e = state[2].cpu()[pg, :, slot].double()
    top, slack = ref.abs().amax(-1), off.amax(-1)
    exp = lambda t: quantised(t[..., None].expand(*t.shape, d))[1].double()  # noqa: E731
    assert bool((exp(top - slack) <= e).all() and (e <= exp(top + slack)).all())
    scale = torch.exp2(e - 127)[..., None]
    err = (stored * scale - ref).abs()
    bound = torch.maximum(2.0 ** -4 * (ref.abs() + off), 2.0 ** -10 * scale) * 1.0001 + off
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("f8", [False, True])
def test_append_edges_of_values(f8):
    # rows of zeros, infinities, NaN, tiny and huge values, without norm and rotation: the write's bits
    d = 64
    rows = torch.zeros(9, 1, d)
    rows[1, 0, 3], rows[2, 0, 3] = 448.0, 449.0
    rows[3] = 2.0 ** -133
    rows[4, 0, 5], rows[5, 0, 7], rows[6, 0, 7] = -3.3e38, float("nan"), float("-inf")
    rows[7] = torch.linspace(-1, 1, d)
    rows[8] = -0.0
    x = rows.to(torch.bfloat16).cuda()
    b = fm.PagedBatch(_i32(0, 9), _i32(9), _i32(0).view(1, 1))
    caches = [fm.fm_cache_new(1, 1, 16, d, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16) for _ in range(2)]
    for c in caches:
        for t in (c.k, c.v, c.k_exp, c.v_exp):
            if t is not None:
                t.view(torch.uint8).zero_()
    out = fm.fm_cache_append(x, x, -x, caches[0], b)
    assert torch.equal(out.nan_to_num(5.0), x.nan_to_num(5.0))
    fm.fm_cache_write(x, -x, caches[1], b)
    a, w = _state(caches[0]), _state(caches[1])
    if f8:
        assert all(torch.equal(p, q) for p, q in zip(a, w))
    else:
        assert torch.equal(caches[0].k.nan_to_num(5.0), caches[1].k.nan_to_num(5.0)) and torch.equal(a[1], w[1])
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("off, kv_len", [((0, 6, 5), (20, 5)), ((0, 3, 9), (20, 5)), ((3, 1, 5), (20, 5)),
                                         ((-4, 3, 5), (20, 5)), ((0, 3, 5), (33, 5)), ((0, 3, 5), (-1, 5)),
                                         ((0, 3, 5), (20, 2 ** 31 - 1))])
@pytest.mark.parametrize("f8", [False, True])
def test_append_flags_what_no_batch_has_and_writes_nothing(off, kv_len, f8):
    s = Setup([32, 20], [3, 2], 2, 64, 16, f8, seed=61)
    before = _state(s.cache)
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16).cuda()
    out = torch.full_like(x, 7.0)
    fm.fm_cache_append(x, x, x, s.cache, fm.PagedBatch(_i32(*off), _i32(*kv_len), s.table), out=out)
    assert fm.fm_device_status() == RANGE
    assert all(torch.equal(a, b) for a, b in zip(before, _state(s.cache))) and (out == 7).all()


def test_append_leaves_out_tokens_without_a_page():
    s = Setup([20, 5], [3, 2], 2, 64, 16, False, seed=62)
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16).cuda()
    for entry in (-1, s.cache.n_pages, 2 ** 31 - 1):
        t = s.table.clone()
        t[0, 1] = entry
        s.cache.k.zero_(), s.cache.v.zero_()
        out = fm.fm_cache_append(x, x, x, s.cache, fm.PagedBatch(s.q_off, s.kv_len, t))
        assert fm.fm_device_status() == RANGE
        assert int(s.cache.k[:, 0, :, 0].sum()) == 2 and int(s.cache.v[:, 0, :, 0].sum()) == 2 and (out == 1).all()
    # more new tokens than keys: the first have no place
    s.cache.k.zero_()
    fm.fm_cache_append(x, x, x, s.cache, fm.PagedBatch(s.q_off, _i32(2, 5), s.table))
    assert fm.fm_device_status() == RANGE
    assert int(s.cache.k[:, 0, :, 0].sum()) == 4


def test_append_in_place_on_a_stream_and_captured():
    s = Setup([70, 33], [1, 1], 2, 128, 16, True, seed=63)
    f, _ = fm.fm_rope_freqs(128, device="cuda")
    qkv = torch.randn(2, 12, 128, generator=s.g).to(torch.bfloat16).cuda()
    work = qkv.clone()

    def step(**kw):
        work.copy_(qkv)
        q, k, v = work.split([8, 2, 2], 1)
        return fm.fm_cache_append(q, k, v, s.cache, s.batch, inv_freq=f, out=q, **kw)

    want = fm.fm_cache_append(*qkv.split([8, 2, 2], 1), s.cache, s.batch, inv_freq=f)
    state = _state(s.cache)
    assert torch.equal(step(), want) and torch.equal(work[:, 8:], qkv[:, 8:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work.copy_(qkv)
    q, k, v = work.split([8, 2, 2], 1)
    got = fm.fm_cache_append(q, k, v, s.cache, s.batch, inv_freq=f, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(state, _state(s.cache)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ((70, 33), (64, 1), (17, 48)):
        s.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        qkv.copy_(torch.randn(qkv.shape, generator=s.g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        a, b = work.clone(), _state(s.cache)
        step()
        assert torch.equal(a, work) and all(torch.equal(x, y) for x, y in zip(b, _state(s.cache)))
    assert fm.fm_device_status() == OK
    # no tokens
    assert fm.fm_cache_append(q[:0], k[:0], v[:0], s.cache, s.batch, inv_freq=f).shape == (0, 8, 128)


def test_append_far_into_a_large_cache():
    # pages whose byte offsets pass 2^32
    for f8 in (False, True):
        s = Setup([200, 64], [1, 5], 8, 128, 64, f8, seed=64, big=70000)
        x = torch.randn(6, 32, 128, generator=s.g).to(torch.bfloat16).cuda()
        fm.fm_cache_append(x[:, :16], x[:, 16:24], x[:, 24:], s.cache, s.batch)
        k, v = fm.fm_cache_read(s.cache, s.kv_off, s.table, 264)
        rows = [199] + list(range(259, 264))
        for got, y in ((k, x[:, 16:24]), (v, x[:, 24:])):
            want = quantised(y.double().cpu())[0] if f8 else y.double().cpu()
            assert torch.equal(got[0, :, rows].double().cpu(), want.transpose(0, 1))
        src, dst = s.table[1, :1].clone(), s.table[0, :1].clone()
        fm.fm_cache_copy(s.cache, src, dst)
        assert all(torch.equal(t[src.long()].view(torch.uint8), t[dst.long()].view(torch.uint8))
                   for t in (s.cache.k, s.cache.v))
        assert fm.fm_device_status() == OK
        del s, k, v


@pytest.mark.parametrize("Hkv, d, page", [(1, 64, 16), (3, 128, 32), (8, 128, 64), (2, 256, 128), (5, 64, 128)])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_copy(Hkv, d, page, f8, n):
    g = torch.Generator().manual_seed(65)
    cache = fm.fm_cache_new(2 * n + 5, Hkv, page, d, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16)
    for t in (cache.k, cache.v, cache.k_exp, cache.v_exp):
        if t is not None:
            b = t.view(torch.uint8)
            b.copy_(torch.randint(0, 256, b.shape, generator=g, dtype=torch.uint8))  # any bytes, NaN among them
    before = _state(cache)
    ids = torch.randperm(2 * n + 5, generator=g).int()
    src, dst = ids[torch.randint(0, n, (n,), generator=g)], ids[n:2 * n].clone()  # a page copied several times
    if n > 2:
        src[2] = dst[2] = -1  # nothing
        src[1] = dst[1]  # a page onto itself
    fm.fm_cache_copy(cache, src.cuda(), dst.cuda())
    assert fm.fm_device_status() == OK
    pairs = dst >= 0
    for a, b in zip(before, _state(cache)):
        a = a.cpu()
        a[dst[pairs].long()] = a[src[pairs].long()]
        assert torch.equal(a, b.cpu())


def test_copy_flags_pages_outside_the_cache():
    cache = fm.fm_cache_new(6, 2, 16, 64)
    cache.k.copy_(torch.arange(6)[:, None, None, None].expand_as(cache.k)), cache.v.zero_()
    for a, b in ((6, 1), (1, 6), (-1, 1), (1, -1), (2 ** 31 - 1, 1), (1, -(2 ** 31)), (-2, -2)):
        fm.fm_cache_copy(cache, _i32(0, a, 2), _i32(3, b, 4))
        assert fm.fm_device_status() == RANGE
        assert cache.k[:, 0, 0, 0].tolist() == [0, 1, 2, 0, 2, 5]
        cache.k.copy_(torch.arange(6)[:, None, None, None].expand_as(cache.k))
    fm.fm_cache_copy(cache, _i32()[:0], _i32()[:0])
    assert fm.fm_device_status() == OK
