"""GPU: the paged cache (written, read back) and the attention of new tokens
over it, against the 64-bit forms of serve_ref."""
import numpy as np
import pytest
import torch

import mask_aware_sparse_gb300 as fm
from serve_ref import assert_paged, paged, quantised

pytestmark = pytest.mark.gpu


class Setup:
    """A cache of sequences with the given keys, pages in a shuffled order, every
    other place of the cache (tails of last pages, unused pages) filled with NaN."""

    def __init__(self, keys, new, Hkv, d, page, f8, seed=0, spare=3, pad=0, big=None):
        self.keys, self.new, self.Hkv, self.d, self.page, self.f8 = keys, new, Hkv, d, page, f8
        g = torch.Generator().manual_seed(seed)
        self.g = g
        width = max(1, max(-(-x // page) for x in keys)) + pad
        n_pages = sum(-(-x // page) for x in keys) + spare
        ids = torch.randperm(n_pages, generator=g)
        if big:  # the same pages at the end of a cache of `big` pages
            ids, n_pages = ids + big - n_pages, big
        self.cache = fm.fm_cache_new(n_pages, Hkv, page, d, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16)
        if not big:
            if f8:
                for t in (self.cache.k, self.cache.v):
                    t.view(torch.uint8).fill_(0x7f)
                for t in (self.cache.k_exp, self.cache.v_exp):
                    t.fill_(255)
            else:
                self.cache.k.fill_(float("nan"))
                self.cache.v.fill_(float("nan"))
        table = torch.full((len(keys), width), -7, dtype=torch.int32)
        at = 0
        for r, x in enumerate(keys):
            n = -(-x // page)
            table[r, :n] = ids[at:at + n]
            at += n
        self.table = table.cuda()
        off = lambda xs: torch.tensor([sum(xs[:i]) for i in range(len(xs) + 1)], dtype=torch.int32).cuda()  # noqa: E731
        self.q_off, self.kv_off = off(new), off(keys)
        self.kv_len = torch.tensor(keys, dtype=torch.int32).cuda()
        self.batch = fm.PagedBatch(self.q_off, self.kv_len, self.table)
        # every key is written: all of them count as new in the call that writes them
        self.k, self.v = (torch.randn(sum(keys), Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
        fm.fm_cache_write(self.k.cuda(), self.v.cuda(), self.cache,
                          fm.PagedBatch(self.kv_off, self.kv_len, self.table))

    def values(self):
        """The cache's keys and values, per sequence (H_kv, L, d) double."""
        out = []
        for x in (self.k, self.v):
            x = x.double()
            x = quantised(x)[0] if self.f8 else x
            out.append([t.transpose(0, 1) for t in x.split(self.keys)])
        return out

    def attend(self, Hq, causal=True, window=0, sinks=0, extra=0, check=True, **kw):
        T = sum(self.new)
        q = torch.randn(T + extra, Hq, self.d, generator=self.g).to(torch.bfloat16)
        scale = self.d ** -0.5
        o, lse = fm.fm_attn_paged(q.cuda(), self.cache, self.batch, scale=scale, causal=causal, window=window,
                                  sinks=sinks, **kw)
        if check:
            k, v = self.values()
            ref = paged(q[:T].double(), k, v, self.q_off.tolist(), self.keys, scale, causal, window, sinks)
            assert_paged(o[:T], lse[:T], ref, self.d)
        assert fm.fm_device_status() == (fm.FM_OK, 0)
        return q, o, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("f8", [False, True])
def test_write_and_read(d, page, f8):
    s = Setup([page * 3 + 5, 1, page, 0, 2 * page - 1], [1, 1, 1, 0, 1], 3, d, page, f8)
    n = sum(s.keys)
    k, v = fm.fm_cache_read(s.cache, s.kv_off, s.table, n + 4,
                            k=torch.full((1, 3, n + 4, d), 7.0, dtype=torch.bfloat16).cuda())
    assert (k[:, :, n:] == 7).all()  # rows behind the last sequence are left as they were
    for got, x in ((k, s.k), (v, s.v)):
        want = quantised(x.double())[0] if f8 else x.double()
        assert torch.equal(got[0, :, :n].double().cpu(), want.transpose(0, 1))
    assert fm.fm_device_status() == (fm.FM_OK, 0)


@pytest.mark.parametrize("d, page, Hkv", [(64, 16, 5), (128, 64, 2), (256, 128, 1)])
@pytest.mark.parametrize("f8", [False, True])
def test_write_and_read_of_many_rows(d, page, Hkv, f8):
    # blocks of many tokens, and one with a few left; rows at an odd 16 bytes
    s = Setup([9001, 3, 0, 2500], [1, 1, 0, 1], Hkv, d, page, f8, seed=24)
    n = sum(s.keys)
    buf = torch.empty(2, Hkv * n * d + 8, dtype=torch.bfloat16).cuda()
    k, v = fm.fm_cache_read(s.cache, s.kv_off, s.table, n, k=buf[0, 8:].view(1, Hkv, n, d),
                            v=buf[1, :-8].view(1, Hkv, n, d))
    for got, x in ((k, s.k), (v, s.v)):
        want = quantised(x.double())[0] if f8 else x.double()
        assert torch.equal(got[0].double().cpu(), want.transpose(0, 1))
    assert fm.fm_device_status() == (fm.FM_OK, 0)


def test_quantisation_edges():
    d = 64
    rows = torch.zeros(12, 1, d)
    rows[1, 0, 3] = 448.0
    rows[2, 0, 3] = 449.0  # bf16 450: one exponent up
    rows[3, 0, :] = 2.0 ** -133  # below the smallest scale
    rows[4, 0, 5] = -3.3e38
    rows[5, 0, 0], rows[5, 0, 1] = 1.0, 2.0 ** -12
    rows[6, 0, 7] = float("nan")
    rows[7, 0, 7] = float("-inf")
    rows[8, 0, :] = torch.linspace(-1, 1, d)
    rows[9, 0, 0] = 0.875 * 2 ** 9
    rows[10] = torch.randn(1, d, generator=torch.Generator().manual_seed(1)) * 1e30
    rows[11] = -0.0
    x = rows.to(torch.bfloat16)
    cache = fm.fm_cache_new(1, 1, 16, d, dtype=torch.float8_e4m3fn)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    b = fm.PagedBatch(i32(0, 12), i32(12), i32(0).view(1, 1))
    fm.fm_cache_write(x.cuda(), (-x).cuda(), cache, b)
    k, v = fm.fm_cache_read(cache, i32(0, 12), b.page_table, 12)
    want, e = quantised(x.double())
    assert torch.equal(cache.k_exp[0, 0, :12].cpu(), e[:, 0])
    for got, w in ((k, want), (v, -want)):
        got = got[0, 0].double().cpu()
        w = w[:, 0].to(torch.bfloat16).double()  # what e4m3 times its scale is beyond bf16's range becomes infinite
        assert torch.equal(torch.isnan(got), torch.isnan(w)) and torch.equal(got.nan_to_num(7), w.nan_to_num(7))


def test_write_takes_views_and_skips_tokens_of_no_sequence():
    s = Setup([40, 23], [3, 2], 2, 128, 16, False)
    before = s.cache.k.clone()
    qkv = torch.randn(8, 6, 128, generator=s.g).to(torch.bfloat16).cuda()
    fm.fm_cache_write(qkv[:, 2:4], qkv[:, 4:6], s.cache, s.batch)  # 5 new tokens, 3 of no sequence
    k, v = fm.fm_cache_read(s.cache, s.kv_off, s.table, 63)
    for i, row in enumerate([37, 38, 39, 40 + 21, 40 + 22]):
        assert torch.equal(k[0, :, row], qkv[i, 2:4]) and torch.equal(v[0, :, row], qkv[i, 4:6])
    assert int((s.cache.k.view(torch.int16) != before.view(torch.int16)).any(-1).any(1).sum()) <= 5
    assert fm.fm_device_status() == (fm.FM_OK, 0)


def test_bad_metadata_is_flagged_and_stays_inside():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    cache = fm.fm_cache_new(4, 2, 16, 64)
    cache.k.zero_(), cache.v.zero_()
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16).cuda()
    q = torch.ones(5, 4, 64, dtype=torch.bfloat16).cuda()
    good = dict(q_off=i32(0, 3, 5), kv_len=i32(20, 5), table=i32(0, 1, 2, 3).view(2, 2))
    for bad in (dict(table=i32(0, 4, 2, 3).view(2, 2)), dict(table=i32(0, -1, 2, 3).view(2, 2)),
                dict(table=i32(0, 2 ** 31 - 1, 2, 3).view(2, 2)), dict(kv_len=i32(33, 5)), dict(kv_len=i32(-1, 5))):
        a = {**good, **bad}
        b = fm.PagedBatch(a["q_off"], a["kv_len"], a["table"])
        fm.fm_cache_write(x, x, cache, b)
        assert fm.fm_device_status() == (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE), bad
        o, lse = fm.fm_attn_paged(q, cache, b, scale=0.1)
        assert fm.fm_device_status() == (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE), bad
        assert torch.isfinite(o[3:]).all()
    for off in (i32(0, 6, 5), i32(0, 3, 9), i32(3, 1, 5), i32(-4, 3, 5)):
        fm.fm_attn_paged(q, cache, fm.PagedBatch(off, good["kv_len"], good["table"]), scale=0.1)
        assert fm.fm_device_status() == (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE), off
    # more new tokens than keys: the first ones see nothing, and have no place to be written to
    b = fm.PagedBatch(i32(0, 3, 5), i32(2, 5), good["table"])
    o, lse = fm.fm_attn_paged(q, cache, b, scale=0.1)
    assert fm.fm_device_status() == (fm.FM_OK, 0)
    assert torch.isneginf(lse[0]).all() and (o[0] == 0).all() and torch.isfinite(lse[1:]).all()
    fm.fm_cache_write(x, x, cache, b)
    assert fm.fm_device_status() == (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE)


def test_overlapping_spans_of_a_large_batch_plan_nothing():
    # descending offsets: five spans of all nine tokens, whose tiles times the CTAs pass 32 bits
    R, Hkv, width = 9, 64, 1000
    cache = fm.fm_cache_new(1, Hkv, 128, 64)
    cache.k.zero_(), cache.v.fill_(1.0)
    kv_len = torch.full((R,), 128 * width, dtype=torch.int32).cuda()
    table = torch.zeros(R, width, dtype=torch.int32).cuda()
    q = torch.zeros(R, 16 * Hkv, 64, dtype=torch.bfloat16).cuda()
    bad = fm.PagedBatch(torch.tensor([0, R] * 5, dtype=torch.int32).cuda(), kv_len, table)
    fm.fm_attn_paged(q, cache, bad, scale=1.0)
    assert fm.fm_device_status() == (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE)
    good = fm.PagedBatch(torch.arange(R + 1, dtype=torch.int32).cuda(), kv_len // 100, table)
    o, lse = fm.fm_attn_paged(q, cache, good, scale=1.0)
    assert (o == 1).all() and float((lse - np.log(1280)).abs().max()) <= 1e-5
    assert fm.fm_device_status() == (fm.FM_OK, 0)


# single tokens: keys of each sequence, heads, head dim, page
STEPS = [
    ([1], 1, 1, 64, 16), ([17], 4, 1, 128, 16), ([64, 65, 63], 8, 8, 128, 64), ([5, 700, 0, 129, 128], 6, 3, 64, 32),
    ([1000, 33], 16, 1, 128, 128), ([3, 300], 8, 2, 256, 16), ([257], 64, 1, 128, 32), ([2500], 5, 1, 64, 64),
    ([31] * 40, 12, 2, 128, 16),
]


@pytest.mark.parametrize("keys, Hq, Hkv, d, page", STEPS)
@pytest.mark.parametrize("f8", [False, True])
def test_single_tokens(keys, Hq, Hkv, d, page, f8):
    s = Setup(keys, [1 if x else 0 for x in keys], Hkv, d, page, f8, pad=2)
    s.attend(Hq)


# chunks: new tokens and keys
CHUNKS = [
    ([3], [3], 4, 2, 64, 16), ([40, 1, 0, 7], [100, 50, 30, 7], 4, 2, 128, 32), ([130], [130], 3, 3, 64, 64),
    ([65, 200], [400, 200], 8, 1, 128, 16), ([33, 2], [64, 1000], 10, 2, 64, 128), ([20, 9], [50, 300], 4, 1, 256, 32),
    ([300], [1111], 8, 2, 128, 64), ([5, 6, 7, 8], [5, 70, 7, 200], 64, 1, 64, 32), ([129], [260], 7, 1, 128, 16),
    ([260, 300], [600, 301], 2, 1, 128, 128), ([257], [257], 1, 1, 64, 16), ([3, 150], [40, 160], 48, 1, 128, 32),
    ([2, 70], [90, 70], 160, 1, 64, 16),
]


@pytest.mark.parametrize("new, keys, Hq, Hkv, d, page", CHUNKS)
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(new, keys, Hq, Hkv, d, page, f8, causal):
    s = Setup(keys, new, Hkv, d, page, f8, seed=2)
    s.attend(Hq, causal=causal)


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (64, 0), (100, 70), (1000, 3), (130, 300)])
@pytest.mark.parametrize("new, keys, G, d", [([1, 1], [900, 20], 4, 128), ([70, 3], [500, 300], 2, 64),
                                             ([300], [700], 4, 128)])
def test_windows(window, sinks, new, keys, G, d):
    s = Setup(keys, new, 2, d, 32, False, seed=3)
    s.attend(2 * G, window=window, sinks=sinks)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("new, keys", [([1, 1], [900, 333]), ([30, 40], [700, 333])])
def test_pages_behind_the_window_may_be_gone(page, f8, new, keys):
    window, sinks = 100, 5
    s = Setup(keys, new, 2, 64, page, f8, seed=22)
    q, o, lse = s.attend(4, window=window, sinks=sinks)
    for r, (n, L) in enumerate(zip(new, keys)):
        lo = L - n - window + 1  # the first key that the first new token sees in its window
        for i in range(s.table.shape[1]):
            if i * page >= sinks and (i + 1) * page <= lo:
                s.table[r, i] = -1 if r else 2 ** 30
    assert int((s.table[:, :5] == -1).sum()) >= 2
    o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=64 ** -0.5, window=window, sinks=sinks)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert fm.fm_device_status() == (fm.FM_OK, 0)


def test_large_window_is_no_window():
    s = Setup([333, 90], [9, 90], 2, 64, 16, True)
    q, o, lse = s.attend(4)
    o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=64 ** -0.5, window=2 ** 31 - 1, sinks=2 ** 31 - 1)
    # the same keys in the same tiles
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("new, keys", [([1, 1, 1], [300, 20, 70]), ([150, 3], [300, 9])])
def test_same_bits_padding_rows_and_views(new, keys):
    s = Setup(keys, new, 2, 128, 32, False, seed=4)
    T = sum(new)
    o = torch.full((T + 3, 4, 128), 9.0, dtype=torch.bfloat16).cuda()
    lse = torch.full((T + 3, 4), 9.0).cuda()
    q, o1, l1 = s.attend(4, extra=3, o=o, lse=lse)
    assert (o1[T:] == 9).all() and (l1[T:] == 9).all()
    # a fused projection's queries, outputs into a wider tensor, a kept workspace
    wide = torch.zeros(T + 3, 8, 128, dtype=torch.bfloat16).cuda()
    wide[:, :4] = q.cuda()
    out = torch.zeros(T + 3, 6, 128, dtype=torch.bfloat16).cuda()
    ws = torch.full((fm.fm_attn_paged_workspace_bytes(s.cache, s.batch, T + 3, 4),), 0xff, dtype=torch.uint8).cuda()
    for _ in range(2):
        o2, l2 = fm.fm_attn_paged(wide[:, :4], s.cache, s.batch, scale=128 ** -0.5, o=out[:, 1:5], ws=ws)
        assert torch.equal(out[:T, 1:5], o1[:T]) and torch.equal(l2[:T], l1[:T])
    assert (out[:, 0] == 0).all() and (out[:, 5] == 0).all() and (out[T:] == 0).all()
    with pytest.raises(ValueError, match="ws"):
        fm.fm_attn_paged(wide[:, :4], s.cache, s.batch, scale=1.0, ws=ws[:-1])


@pytest.mark.parametrize("new, keys, d", [([1], [3000], 128), ([70], [3000], 128), ([90], [2500], 64)])
def test_a_workspace_at_any_16_byte_boundary(new, keys, d):
    # divided units leave parts there
    s = Setup(keys, new, 2, d, 32, False, seed=21)
    T = new[0]
    need = fm.fm_attn_paged_workspace_bytes(s.cache, s.batch, T, 8)
    buf = torch.full((need + 512,), 0x5a, dtype=torch.uint8).cuda()
    q, o, lse = s.attend(8)
    for at in (16, 48, 240):
        o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=d ** -0.5, ws=buf[at:at + need])
        assert torch.equal(o2, o) and torch.equal(l2, lse)
        assert (buf[:at] == 0x5a).all() and (buf[at + need:] == 0x5a).all()


def test_quantised_is_the_cache_read_back():
    # an e4m3 cache gives what its bf16 copy gives, up to the order of the same sums
    s = Setup([500, 77], [40, 1], 2, 128, 32, True, seed=5)
    q, o, lse = s.attend(8)
    copy = fm.fm_cache_new(s.cache.k.shape[0], 2, 32, 128)
    n = sum(s.keys)
    k, v = fm.fm_cache_read(s.cache, s.kv_off, s.table, n)
    fm.fm_cache_write(k[0].transpose(0, 1), v[0].transpose(0, 1), copy, fm.PagedBatch(s.kv_off, s.kv_len, s.table))
    o2, l2 = fm.fm_attn_paged(q.cuda(), copy, s.batch, scale=128 ** -0.5)
    k, v = s.values()
    ref = paged(q.double(), k, v, s.q_off.tolist(), s.keys, 128 ** -0.5, True, 0, 0)
    assert_paged(o2, l2, ref, 128)
    assert float((lse - l2).abs().max()) <= 1e-4


@pytest.mark.parametrize("new", [[1, 1], [60, 20]])
@pytest.mark.parametrize("f8", [False, True])
def test_large_and_outlying_values(new, f8):
    # rows of very different scales: running maxima that move, exponents far apart
    s = Setup([300, 140], new, 2, 64, 16, f8, seed=6)
    m = torch.exp2(torch.randint(-6, 7, (sum(s.keys), 2, 1), generator=s.g).double())
    s.k, s.v = (s.k.double() * m).to(torch.bfloat16), (s.v.double() * m * 2.0 ** 20).to(torch.bfloat16)
    fm.fm_cache_write(s.k.cuda(), s.v.cuda(), s.cache, fm.PagedBatch(s.kv_off, s.kv_len, s.table))
    s.attend(4)


def test_subnormal_queries_of_large_quantised_keys():
    s = Setup([90, 33], [1, 1], 2, 64, 16, True, seed=23)
    s.k = (s.k.double() * 2.0 ** 118).to(torch.bfloat16)
    fm.fm_cache_write(s.k.cuda(), s.v.cuda(), s.cache, fm.PagedBatch(s.kv_off, s.kv_len, s.table))
    q = (torch.randn(2, 4, 64, generator=s.g).double() * 2.0 ** -129).to(torch.bfloat16)
    o, lse = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=512.0)
    k, v = s.values()
    assert_paged(o, lse, paged(q.double(), k, v, s.q_off.tolist(), s.keys, 512.0, True, 0, 0), 64)


def test_long_cache_offsets_beyond_32_bits():
    # pages at the end of a cache whose byte offsets pass 2^32
    for f8 in (False, True):
        s = Setup([200, 64], [1, 5], 8, 128, 64, f8, seed=7, big=70000)
        assert s.cache.k.numel() * s.cache.k.element_size() > 2 ** 32
        s.attend(16)
        k, _ = fm.fm_cache_read(s.cache, s.kv_off, s.table, 264)
        want = quantised(s.k.double())[0] if f8 else s.k.double()
        assert torch.equal(k[0].double().cpu(), want.transpose(0, 1))
        del s, k


def test_many_sequences_and_shared_pages():
    # 1500 sequences (more than a block plans at once); all read one prefix page
    R, page = 1500, 16
    g = torch.Generator().manual_seed(8)
    cache = fm.fm_cache_new(R + 1, 1, page, 64)
    kv = torch.randn(2, R + 1, 1, page, 64, generator=g).to(torch.bfloat16)
    cache.k.copy_(kv[0]), cache.v.copy_(kv[1])
    keys = torch.randint(17, 33, (R,), generator=g)
    new = (torch.rand(R, generator=g) < 0.8).int()
    table = torch.stack((torch.zeros(R, dtype=torch.int32), torch.arange(1, R + 1, dtype=torch.int32)), 1)
    q_off = torch.cat((torch.zeros(1, dtype=torch.int32), new.cumsum(0).int()))
    T = int(q_off[-1])
    q = torch.randn(T, 2, 64, generator=g).to(torch.bfloat16)
    batch = fm.PagedBatch(q_off.cuda(), keys.int().cuda(), table.cuda())
    o, lse = fm.fm_attn_paged(q.cuda(), cache, batch, scale=0.125)
    assert fm.fm_device_status() == (fm.FM_OK, 0)
    seq = lambda c, r: torch.cat((c[0, 0], c[r + 1, 0]))[: int(keys[r])].double()[None]  # noqa: E731
    ref = paged(q.double(), [seq(kv[0], r) for r in range(R)], [seq(kv[1], r) for r in range(R)], q_off.tolist(),
                keys.tolist(), 0.125, True, 0, 0)
    assert_paged(o, lse, ref, 64)


def test_streams_and_graph_replay():
    # two calls at once on two streams; a captured step replayed with other lengths
    a = Setup([700, 90], [1, 1], 2, 128, 16, False, seed=9)
    b = Setup([300, 450], [100, 30], 2, 64, 32, True, seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qa, oa, la = a.attend(8)
    qb, ob, lb = b.attend(4)
    qa, qb = qa.cuda(), qb.cuda()
    torch.cuda.synchronize()
    for _ in range(3):
        o1, l1 = fm.fm_attn_paged(qa, a.cache, a.batch, scale=128 ** -0.5)
        o2, l2 = torch.empty_like(ob), torch.empty_like(lb)
        ws = torch.empty(fm.fm_attn_paged_workspace_bytes(b.cache, b.batch, 130, 4), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        fm.fm_attn_paged(qa, a.cache, a.batch, scale=128 ** -0.5, o=o1, lse=l1)
        fm.fm_attn_paged(qb, b.cache, b.batch, scale=64 ** -0.5, o=o2, lse=l2, ws=ws, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o1, oa) and torch.equal(o2, ob) and torch.equal(l2, lb)
    # capture: write one token of each sequence, then attend
    kv = torch.randn(2, 2, 2, 128, generator=a.g).to(torch.bfloat16).cuda()
    o, lse = torch.empty_like(oa), torch.empty_like(la)
    ws = torch.empty(fm.fm_attn_paged_workspace_bytes(a.cache, a.batch, 2, 8), dtype=torch.uint8, device="cuda")

    def step():
        fm.fm_cache_write(kv[0], kv[1], a.cache, a.batch)
        fm.fm_attn_paged(qa, a.cache, a.batch, scale=128 ** -0.5, o=o, lse=lse, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([700, 90], [650, 70], [1, 33]):
        a.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        kv.copy_(torch.randn(kv.shape, generator=a.g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        k, _ = fm.fm_cache_read(a.cache, torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32).cuda(), a.table,
                                sum(lens))
        assert torch.equal(k[0, :, lens[0] - 1], kv[0, 0]) and torch.equal(k[0, :, -1], kv[0, 1])
    assert fm.fm_device_status() == (fm.FM_OK, 0)


def test_a_served_sequence_is_the_trained_one():
    # norm + rotation, cache write and attention, chunk by chunk and token by
    # token, against one flashmask_attention over the whole packed sequence
    from workloads import masks

    Hq, Hkv, d, N, page = 8, 2, 128, 200, 16
    g = torch.Generator().manual_seed(11)
    qkv = torch.randn(1, N, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (t.transpose(1, 2) for t in qkv.split([Hq, Hkv, Hkv], 2))
    f, sc = fm.fm_rope_freqs(d, kind="yarn", factor=2.0, orig_len=128, device="cuda")
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()
    spec = fm.QKNormRope(positions=pos, inv_freq=f, rot_scale=sc, q_weight=w[0], k_weight=w[1])
    for window, sinks in ((0, 0), (64, 4)):
        vec = masks.sliding_window(N, window, sinks) if window else masks.causal_documents([N], N)
        vec = [torch.from_numpy(np.ascontiguousarray(x[None])).cuda() for x in vec]
        want = fm.flashmask_attention(q, k, v, *vec, causal=True, qk=spec)[0].transpose(0, 1)  # (N, H_q, d)
        cache = fm.fm_cache_new(-(-N // page), Hkv, page, d)
        q_off, kv_len = torch.zeros(2, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
        batch = fm.PagedBatch(q_off, kv_len, torch.randperm(-(-N // page), generator=g).int()[None].cuda())
        at = 0
        for n in [50, 77, 1, 1, 3, 60] + [1] * 8:
            q_off[1] = n
            kv_len[0] = at + n
            part = [t[:, :, at:at + n] for t in (q, k, v)]
            out = [torch.empty(n, t.shape[1], d, dtype=torch.bfloat16, device="cuda") for t in part[:2]]
            fm.fm_qk_norm_rope(part[0], part[1], positions=pos[at:at + n], inv_freq=f, rot_scale=sc, q_weight=w[0],
                               k_weight=w[1], out=tuple(t.transpose(0, 1)[None] for t in out))
            fm.fm_cache_write(out[1], part[2][0].transpose(0, 1), cache, batch)
            o, _ = fm.fm_attn_paged(out[0], cache, batch, scale=d ** -0.5, window=window, sinks=sinks)
            # both round P once and O once: each within 2^-7 of sum p |v|, at most the largest |v|
            err = (o.double() - want[at:at + n].double()).abs().max()
            assert float(err) <= 2 * 2.0 ** -7 * float(v.abs().max())
            rel = (o.double() - want[at:at + n].double()).norm() / want[at:at + n].double().norm()
            assert float(rel) <= 2 * 2.0 ** -7
            at += n
        assert at == N
    assert fm.fm_device_status() == (fm.FM_OK, 0)


@pytest.mark.parametrize("d, f8", [(64, True), (128, False), (128, True)])
def test_many_chunks_of_ragged_lengths(d, f8):
    # more sequences than a CTA plans for by itself: chunks of every size beside single tokens
    g = torch.Generator().manual_seed(12)
    new = torch.randint(0, 60, (45,), generator=g).tolist()
    new[3], new[7], new[20] = 400, 1, 0
    keys = [n + int(x) for n, x in zip(new, torch.randint(0, 300, (45,), generator=g))]
    s = Setup(keys, new, 2, d, 32, f8, seed=13)
    s.attend(6)


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("d, Hq, Hkv, n", [(128, 8, 2, 1300), (64, 2, 2, 2000)])
def test_a_prompt_over_itself(d, Hq, Hkv, n, window):
    # whole units, dealt largest first: one per CTA and more
    s = Setup([n], [n], Hkv, d, 64, False, seed=14)
    s.attend(Hq, window=window, sinks=3 if window else 0)
    s = Setup([n, 77], [n, 50], Hkv, d, 64, False, seed=15)
    s.attend(Hq, window=window)


def test_one_long_sequence_among_short_ones():
    s = Setup([4000] + [20] * 30, [1] * 31, 2, 64, 16, False, seed=16)
    s.attend(8)
    s = Setup([3000] + [40] * 20, [40] + [30] * 20, 1, 64, 16, True, seed=17)
    s.attend(4)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 50])
def test_new_tokens_without_keys(n, causal):
    s = Setup([64, 30], [0, 0], 2, 64, 16, False, seed=18)
    kv_len = torch.tensor([0, 30], dtype=torch.int32).cuda()
    b = fm.PagedBatch(torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda(), kv_len, s.table)
    q = torch.randn(2 * n, 4, 64, generator=s.g).to(torch.bfloat16).cuda()
    o, lse = fm.fm_attn_paged(q, s.cache, b, scale=0.125, causal=causal)
    assert (o[:n] == 0).all() and torch.isneginf(lse[:n]).all()
    k, v = s.values()
    ref = paged(q[n:].double().cpu(), [k[1]], [v[1]], [0, n], [30], 0.125, causal, 0, 0)
    assert_paged(o[n:], lse[n:], ref, 64)
    # no tokens at all
    o, lse = fm.fm_attn_paged(q[:0], s.cache, b, scale=0.125)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    fm.fm_cache_write(q[:0, :2], q[:0, :2], s.cache, b)
    assert fm.fm_device_status() == (fm.FM_OK, 0)


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 30, 60]])
@pytest.mark.parametrize("f8", [False, True])
def test_a_visible_nan_stays_in_its_sequence(new, f8):
    s = Setup([100, 90, 200], new, 2, 64, 16, f8, seed=19)
    q, o, lse = s.attend(4)
    for which in (s.k, s.v):
        bad = which.clone()
        bad[100 + 5] = float("nan")  # key 5 of the second sequence
        fm.fm_cache_write(*((bad.cuda(), s.v.cuda()) if which is s.k else (s.k.cuda(), bad.cuda())), s.cache,
                          fm.PagedBatch(s.kv_off, s.kv_len, s.table))
        o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=64 ** -0.5)
        a, b = s.q_off.tolist()[1:3]
        assert torch.isnan(o2[a:b]).all()
        for part in (slice(0, a), slice(b, None)):
            assert torch.equal(o2[part], o[part]) and torch.equal(l2[part], lse[part])


def test_a_given_stream_owns_what_a_call_allocates():
    # a slow stream: memory that the call's outputs and workspace came from is not
    # handed out again before the stream has passed
    s = Setup([3000], [1], 2, 128, 16, False, seed=20)
    q, o, lse = s.attend(8)
    q = q.cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    outs = [fm.fm_attn_paged(q, s.cache, s.batch, scale=128 ** -0.5, stream=side) for _ in range(3)]
    junk = [torch.full((1 << 22,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(40)]
    side.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)
    del junk


def test_arguments_refused():
    s = Setup([20], [2], 2, 64, 16, False)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16).cuda()
    for kw in (dict(window=-1), dict(sinks=-1), dict(window=-(2 ** 40)), dict(o=q.float()), dict(o=q[:1]),
               dict(lse=torch.zeros(2, 4)), dict(lse=torch.zeros(4, 2).cuda()), dict(ws=torch.zeros(8).cuda()),
               dict(o=q[:, :1].expand(2, 4, 64))):
        with pytest.raises(ValueError):
            fm.fm_attn_paged(q, s.cache, s.batch, scale=0.1, **kw)
    for bad in (q[:, :3], q[..., :32], q.float(), q[0]):
        with pytest.raises((ValueError, fm.FMError)):
            fm.fm_attn_paged(bad, s.cache, s.batch, scale=0.1)
    for kw in (dict(scale=0.0), dict(scale=0.1, causal=False, window=3), dict(scale=float("nan"))):
        with pytest.raises(fm.FMError):
            fm.fm_attn_paged(q, s.cache, s.batch, **kw)
    with pytest.raises(ValueError):
        fm.fm_cache_read(s.cache, s.kv_off, s.table, -1)
    with pytest.raises(ValueError):
        fm.fm_cache_write(q, q[:1], s.cache, s.batch)
    # broadcast queries (a stride of zero) are read like any others
    one = torch.randn(1, 1, 64, generator=s.g).to(torch.bfloat16).cuda()
    a = fm.fm_attn_paged(one.expand(2, 4, 64), s.cache, s.batch, scale=0.1)
    b = fm.fm_attn_paged(one.expand(2, 4, 64).contiguous(), s.cache, s.batch, scale=0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    big = fm.PagedBatch(torch.tensor([0, 20], dtype=torch.int32).cuda(), s.kv_len, s.table)
    a = fm.fm_attn_paged(one.expand(20, 4, 64), s.cache, big, scale=0.1)
    b = fm.fm_attn_paged(one.expand(20, 4, 64).contiguous(), s.cache, big, scale=0.1)
    assert float((a[0].float() - b[0].float()).abs().max()) <= 2 ** -6 * float(s.v.abs().max())
