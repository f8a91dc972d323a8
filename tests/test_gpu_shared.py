"""GPU: attention of sequences that share prefixes, against the 64-bit forms of serve_ref:
each sequence over all of its keys, whoever holds them. Bounds are those of the attention
over the paged cache (a weight rounded once to 2^-8 of it, O once, scores in 32 bits):
joining parts adds 32-bit roundings, which the factor of 2 percent on them covers."""
import pytest
import torch

import mask_aware_sparse_gb300 as fm
from serve_ref import assert_paged, paged, quantised

pytestmark = pytest.mark.gpu
RANGE = (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE)
OK = (fm.FM_OK, 0)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _off(xs):
    return _i32([sum(xs[:i]) for i in range(len(xs) + 1)])


class Groups:
    """A cache of groups of sequences: prefix[g] keys that are the same for all of group
    g, rest[g] = keys of each sequence behind them, new[g] = new tokens of each. Pages in a
    shuffled order, everything else in the cache NaN, the table -7 where nothing is, and as
    wide as it has to be for calls of Hq heads to share (whether they do goes by its width)."""

    def __init__(self, prefix, rest, new, Hkv, d, page, f8, seed=0, pad=0, Hq=None):
        self.prefix, self.Hkv, self.d, self.page, self.f8 = prefix, Hkv, d, page, f8
        self.g = g = torch.Generator().manual_seed(seed)
        self.sizes = [len(x) for x in rest]
        self.keys = [P + x for P, xs in zip(prefix, rest) for x in xs]
        self.new = [x for xs in new for x in xs]
        R, up = len(self.keys), lambda x: -(-x // page)
        whole = [P // page for P in prefix]
        count = sum(w for w, xs in zip(whole, rest) if xs) + sum(up(P + x) - P // page for P, xs in zip(prefix, rest) for x in xs)
        ids = torch.randperm(count + 3, generator=g).int()
        self.cache = fm.fm_cache_new(count + 3, Hkv, page, d, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16)
        for t in (self.cache.k, self.cache.v):
            t.view(torch.uint8).fill_(0x7f) if f8 else t.fill_(float("nan"))
        for t in (self.cache.k_exp, self.cache.v_exp):
            if f8:
                t.fill_(255)
        table = torch.full((R, max([1] + [up(x) for x in self.keys]) + pad), -7, dtype=torch.int32)
        rows = [torch.randn(2, P, Hkv, d, generator=g).to(torch.bfloat16) for P in prefix]
        self.rows, at, r = [], 0, 0
        for i, xs in enumerate(rest):
            w = whole[i]
            if xs:
                shared, at = ids[at:at + w], at + w
            for x in xs:
                n = up(prefix[i] + x)
                table[r, :w] = shared
                table[r, w:n] = ids[at:at + n - w]
                at += n - w
                self.rows.append(torch.cat((rows[i], torch.randn(2, x, Hkv, d, generator=g).to(torch.bfloat16)), 1))
                r += 1
        self.table = table.cuda()
        self.write()
        self.q_off, self.kv_len = _off(self.new), _i32(self.keys)
        self.batch = fm.PagedBatch(self.q_off, self.kv_len, self.table)
        self.seq_off, self.prefix_len = _off(self.sizes), _i32(prefix)
        self.shared = fm.SharedPrefix(self.seq_off, self.prefix_len)
        while Hq and not self.shares(Hq):
            self.table = torch.nn.functional.pad(self.table, (0, self.table.shape[1]), value=-7)
            self.batch = fm.PagedBatch(self.q_off, self.kv_len, self.table)

    def shares(self, Hq):
        T = sum(self.new)
        return (fm.fm_attn_shared_workspace_bytes(self.cache, self.batch, self.shared, T, Hq)
                > fm.fm_attn_paged_workspace_bytes(self.cache, self.batch, T, Hq))

    def write(self):
        """Shared pages by each group's first sequence, then each sequence's own."""
        firsts = [sum(self.sizes[:i]) for i, n in enumerate(self.sizes) if n]
        group = [i for i, n in enumerate(self.sizes) for _ in range(n)]
        for first in (True, False):
            seqs = [r for r in range(len(self.keys)) if (r in firsts) == first]
            skip = [0 if first else self.prefix[group[r]] // self.page * self.page for r in seqs]
            n = [self.keys[r] - x for r, x in zip(seqs, skip)]
            if not seqs or not sum(n):
                continue
            kv = torch.cat([self.rows[r][:, x:] for r, x in zip(seqs, skip)], 1).cuda()
            fm.fm_cache_write(kv[0], kv[1], self.cache,
                              fm.PagedBatch(_off(n), _i32([self.keys[r] for r in seqs]), self.table[seqs].contiguous()))
        assert fm.fm_device_status() == OK

    def reference(self, q, scale, causal):
        k, v = ([(quantised(x[i].double())[0] if self.f8 else x[i].double()).transpose(0, 1) for x in self.rows]
                for i in range(2))
        return paged(q.double(), k, v, self.q_off.tolist(), self.keys, scale, causal, 0, 0)

    def attend(self, Hq, causal=True, extra=0, **kw):
        T = sum(self.new)
        q = torch.randn(T + extra, Hq, self.d, generator=self.g).to(torch.bfloat16)
        scale = self.d ** -0.5
        o, lse = fm.fm_attn_shared(q.cuda(), self.cache, self.batch, self.shared, scale=scale, causal=causal, **kw)
        assert fm.fm_device_status() == OK
        assert_paged(o[:T], lse[:T], self.reference(q[:T], scale, causal), self.d)
        return q, o, lse


def ones(rest):
    return [[1] * len(xs) for xs in rest]


# prefix, rest, Hq, Hkv, d, page; a token a sequence
STEPS = [
    ([100], [[5, 40]], 4, 1, 64, 16),
    ([1021], [[1, 40]], 32, 8, 128, 16),
    ([96], [[1, 33, 64]], 8, 2, 128, 32),  # whole pages
    ([31, 64, 500, 0], [[3, 60], [1], [200, 9, 77, 1], [50, 20]], 6, 3, 64, 32),  # part of a page, a group of one, nothing shared
    ([700], [[10, 300, 40, 7, 90, 1, 33, 64]], 8, 2, 128, 64),
    ([900, 333], [[20] * 9, [31, 1, 5, 160, 2, 7, 9]], 16, 2, 128, 16),
    ([2000], [[50] * 40], 8, 1, 128, 128),
    ([600], [[40, 3, 90]], 8, 2, 256, 16),
    ([1500], [[130] * 12], 8, 1, 256, 64),
    ([300, 40], [[1] * 20, [9] * 30], 4, 2, 64, 128),
    ([257, 1000], [[33] * 7, []], 5, 1, 64, 16),  # a group of none
    ([1000], [[17] * 70], 2, 2, 64, 32),
    ([5000], [[1, 2, 3]], 64, 1, 128, 32),
]


@pytest.mark.parametrize("prefix, rest, Hq, Hkv, d, page", STEPS)
@pytest.mark.parametrize("f8", [False, True])
def test_steps(prefix, rest, Hq, Hkv, d, page, f8):
    s = Groups(prefix, rest, ones(rest), Hkv, d, page, f8, seed=70, pad=2)
    q, o, lse = s.attend(Hq)
    s = Groups(prefix, rest, ones(rest), Hkv, d, page, f8, seed=70, pad=2, Hq=Hq)
    assert s.shares(Hq)
    s.attend(Hq)
    s.attend(Hq, causal=False)


# prefix, rest, new, Hq, Hkv, d, page
MANY = [
    ([200], [[9, 30, 20]], [[4, 5, 3]], 4, 2, 64, 16),  # a few tokens each
    ([700, 90], [[40, 8], [33, 17, 9]], [[5, 2], [0, 7, 1]], 8, 2, 128, 32),
    ([1000], [[60, 70, 35, 90]], [[20, 31, 33, 25]], 8, 2, 128, 64),  # chunks
    ([130, 513], [[40] * 3, [200, 77]], [[40, 1, 33], [30, 0]], 6, 2, 64, 16),
    ([300], [[50, 20, 31]], [[50, 20, 31]], 4, 1, 256, 32),  # all that is not shared is new
    ([64, 3000], [[64, 90], [128, 300]], [[60, 50], [40, 70]], 5, 1, 128, 128),
    ([400], [[30] * 50], [[3, 30] * 25], 4, 2, 64, 32),  # more sequences than a CTA plans for by itself
    ([500], [[300, 200]], [[250, 190]], 4, 2, 128, 64),  # long chunks: as if nothing were shared
    ([77], [[40, 20, 60]], [[9, 20, 11]], 48, 1, 128, 16),
    ([77], [[6, 7, 1]], [[2, 3, 1]], 160, 1, 64, 16),
]


@pytest.mark.parametrize("prefix, rest, new, Hq, Hkv, d, page", MANY)
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens(prefix, rest, new, Hq, Hkv, d, page, f8, causal):
    for share in (False, True):
        s = Groups(prefix, rest, new, Hkv, d, page, f8, seed=71, Hq=Hq if share else None)
        s.attend(Hq, causal=causal)


@pytest.mark.parametrize("f8", [False, True])
def test_many_sequences(f8):
    # planned by a kernel of its own: more sequences than a block plans for, groups of every size
    g = torch.Generator().manual_seed(72)
    sizes = [1, 150, 0, 7, 200, 3]
    rest = [torch.randint(1, 60, (n,), generator=g).tolist() for n in sizes]
    new = [[int(x) for x in (torch.rand(n, generator=g) < 0.8)] for n in sizes]
    s = Groups([40, 300, 20, 0, 97, 16], rest, new, 2, 64, 16, f8, seed=73, Hq=4)
    s.attend(4)
    rest = [[70] * n for n in sizes]
    s = Groups([40, 300, 20, 0, 97, 16], rest, [[int(1 + x) for x in 40 * torch.rand(n, generator=g)] for n in sizes], 2, 128,
               32, f8, seed=74, Hq=4)
    s.attend(4)


@pytest.mark.parametrize("new", [[[0, 1, 1], [1, 0]], [[0, 30, 20], [25, 0]]])
def test_sequences_out_of_use(new):
    # no new tokens: their rows of the table may hold anything, the first one's too, and so may their lengths
    s = Groups([100, 64], [[40, 50, 60], [30, 35]], new, 2, 128, 16, False, seed=75, Hq=8)
    q, o, lse = s.attend(8)
    for r in (0, 4):
        s.table[r] = -1 if r else 2 ** 30
        s.kv_len[r] = 0
    o2, l2 = fm.fm_attn_shared(q.cuda(), s.cache, s.batch, s.shared, scale=128 ** -0.5)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("new, Hq", [([[1, 1, 1], [1, 1]], 8), ([[20, 30, 9], [25, 3]], 8), ([[1] * 3, [1] * 2], 64)])
def test_same_bits_padding_rows_and_views(new, Hq):
    s = Groups([300, 90], [[40, 50, 60], [30, 35]], new, 2, 128, 32, False, seed=76, Hq=Hq)
    T = sum(s.new)
    o = torch.full((T + 3, Hq, 128), 9.0, dtype=torch.bfloat16).cuda()
    lse = torch.full((T + 3, Hq), 9.0).cuda()
    q, o1, l1 = s.attend(Hq, extra=3, o=o, lse=lse)
    assert (o1[T:] == 9).all() and (l1[T:] == 9).all()
    wide = torch.zeros(T + 3, Hq + 4, 128, dtype=torch.bfloat16).cuda()
    wide[:, :Hq] = q.cuda()
    out = torch.zeros(T + 3, Hq + 2, 128, dtype=torch.bfloat16).cuda()
    need = fm.fm_attn_shared_workspace_bytes(s.cache, s.batch, s.shared, T + 3, Hq)
    buf = torch.full((need + 512,), 0xff, dtype=torch.uint8).cuda()
    for at in (0, 16, 240):
        o2, l2 = fm.fm_attn_shared(wide[:, :Hq], s.cache, s.batch, s.shared, scale=128 ** -0.5, o=out[:, 1:-1],
                                   ws=buf[at:at + need])
        assert torch.equal(out[:T, 1:-1], o1[:T]) and torch.equal(l2[:T], l1[:T])
        assert (buf[:at] == 0xff).all() and (buf[at + need:] == 0xff).all()
    assert (out[:, 0] == 0).all() and (out[:, -1] == 0).all() and (out[T:] == 0).all()
    with pytest.raises(ValueError, match="ws"):
        fm.fm_attn_shared(wide[:, :Hq], s.cache, s.batch, s.shared, scale=1.0, ws=buf[:need - 1])
    # broadcast queries (a stride of zero) are read like any others
    one = torch.randn(1, 1, 128, generator=s.g).to(torch.bfloat16).cuda()
    a = fm.fm_attn_shared(one.expand(T, Hq, 128), s.cache, s.batch, s.shared, scale=0.1)
    b = fm.fm_attn_shared(one.expand(T, Hq, 128).contiguous(), s.cache, s.batch, s.shared, scale=0.1)
    assert float((a[0].float() - b[0].float()).abs().max()) <= 2 ** -6 * max(float(x[1].abs().max()) for x in s.rows)
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("new, Hq", [([[1, 1, 1], [1, 1]], 4), ([[1, 1, 1], [1, 1]], 64), ([[20, 30, 9], [25, 3]], 8)])
def test_prefixes_as_long_as_their_sequences(new, Hq):
    # all keys shared: seen by all (no causal mask), and, causal, with nothing between them and the new tokens
    s = Groups([160, 64], [[0, 0, 0], [0, 0]], new, 2, 64, 16, False, seed=86, Hq=Hq)
    s.attend(Hq, causal=False)
    s = Groups([160, 64], new, new, 2, 64, 16, False, seed=87, Hq=Hq)
    s.attend(Hq)


@pytest.mark.parametrize("n, Hq", [(3, 4), (3, 64), (20, 8)])
def test_more_new_tokens_than_keys_behind_no_prefix(n, Hq):
    # the first new tokens see nothing, which is no error, as without groups
    s = Groups([0], [[64, 30, 2]], [[n, n, n]], 2, 64, 16, False, seed=88, Hq=Hq)
    s.kv_len[2] = 2
    q = torch.randn(3 * n, Hq, 64, generator=s.g).to(torch.bfloat16).cuda()
    o, lse = fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=0.125)
    assert fm.fm_device_status() == OK
    assert (o[2 * n:3 * n - 2] == 0).all() and torch.isneginf(lse[2 * n:3 * n - 2]).all()
    assert_paged(o, lse, s.reference(q.cpu(), 0.125, True), 64)


@pytest.mark.parametrize("d, f8", [(64, False), (128, True), (256, False)])
def test_the_workspace_is_enough_for_queries_of_any_strides(d, f8):
    # which kernels run, and whether the call shares, goes by the queries' strides too: for every size the
    # workspace covers both (a broadcast's kernels need other parts)
    for T, R, width in ((6, 6, 4), (6, 6, 4000), (120, 6, 40), (120, 6, 400), (120, 6, 4000), (1300, 6, 2000)):
        cache = fm.fm_cache_new(1, 2, 16, d, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16)
        for t in (cache.k, cache.v, cache.k_exp, cache.v_exp):
            if t is not None:
                t.view(torch.uint8).fill_(1)
        batch = fm.PagedBatch(_off([T // R] * R), _i32([16] * R), torch.zeros(R, width, dtype=torch.int32).cuda())
        shared = fm.SharedPrefix(_i32([0, R]), _i32([0]))
        need = fm.fm_attn_shared_workspace_bytes(cache, batch, shared, T, 8)
        buf = torch.full((need + 512,), 0x5a, dtype=torch.uint8).cuda()
        one = torch.randn(1, 1, d).to(torch.bfloat16).cuda()
        for q in (one.expand(T, 8, d), one.expand(T, 8, d).contiguous()):
            fm.fm_attn_shared(q, cache, batch, shared, scale=0.1, ws=buf[256:256 + need], causal=False)
            assert fm.fm_device_status() == OK
            assert (buf[:256] == 0x5a).all() and (buf[256 + need:] == 0x5a).all()


def test_no_tokens():
    s = Groups([100], [[40, 50]], [[0, 0]], 2, 64, 16, False, seed=77, pad=5000)
    assert fm.fm_attn_shared_workspace_bytes(s.cache, s.batch, s.shared, 5, 4) > fm.fm_attn_paged_workspace_bytes(s.cache, s.batch, 5, 4)
    q = torch.randn(5, 4, 64, generator=s.g).to(torch.bfloat16).cuda()
    o, lse = fm.fm_attn_shared(q[:0], s.cache, s.batch, s.shared, scale=0.125)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = torch.full_like(q, 3.0), torch.full((5, 4), 3.0).cuda()
    fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=0.125, o=o, lse=lse)  # tokens of no sequence
    assert (o == 3).all() and (lse == 3).all()
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("new", [[[1, 1, 1], [1, 1]], [[30, 20, 31], [25, 40]]])
@pytest.mark.parametrize("f8", [False, True])
def test_large_and_outlying_values(new, f8):
    # rows of very different scales, in the prefix and behind it: parts whose maxima are far apart
    s = Groups([300, 140], [[40, 50, 60], [64, 45]], new, 2, 64, 16, f8, seed=78, Hq=4)
    group = [0, 0, 0, 1, 1]
    m = [torch.exp2(torch.randint(-6, 7, (1, P, 2, 1), generator=s.g).double()) for P in s.prefix]
    for r, x in enumerate(s.rows):
        P = s.prefix[group[r]]
        more = torch.exp2(torch.randint(-6, 7, (1, x.shape[1] - P, 2, 1), generator=s.g).double())
        y = x.double() * torch.cat((m[group[r]], more), 1)
        y[1] *= 2.0 ** 20
        s.rows[r] = y.to(torch.bfloat16)
    s.write()
    s.attend(4)


@pytest.mark.parametrize("new", [[[1, 1, 1], [1, 1]], [[30, 20, 31], [25, 40]]])
@pytest.mark.parametrize("f8", [False, True])
def test_a_visible_nan_stays_in_its_group_or_sequence(new, f8):
    s = Groups([100, 64], [[40, 50, 60], [64, 45]], new, 2, 64, 16, f8, seed=79, Hq=4)
    q, o, lse = s.attend(4)
    clean = [x.clone() for x in s.rows]
    off = s.q_off.tolist()
    for seqs, at in (((0, 1, 2), 5), ((4,), 64 + 3), ((1,), 98), ((0,), 101)):  # the prefix; a sequence's own keys
        for which in (0, 1):
            s.rows = [x.clone() for x in clean]
            for r in seqs:
                s.rows[r][which, at] = float("nan")
            s.write()
            o2, l2 = fm.fm_attn_shared(q.cuda(), s.cache, s.batch, s.shared, scale=64 ** -0.5)
            for r in range(5):
                part = slice(off[r], off[r + 1])
                if r in seqs:
                    assert torch.isnan(o2[part]).all()
                else:
                    assert torch.equal(o2[part], o[part]) and torch.equal(l2[part], lse[part])
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("new, Hq", [([[1, 1, 1], [1, 1]], 4), ([[1, 1, 1], [1, 1]], 64), ([[20, 30, 9], [25, 3]], 8)])
def test_what_no_batch_has_is_flagged(new, Hq):
    s = Groups([100, 64], [[40, 50, 60], [30, 35]], new, 2, 64, 16, False, seed=80, Hq=Hq)
    q, o, lse = s.attend(Hq)
    q = q.cuda()
    size = s.table.shape[1] * 16
    n = s.new
    for seq_off, prefix in (((0, 3, 4), (100, 64)), ((0, 6, 5), (100, 64)), ((1, 3, 5), (100, 64)), ((0, 3, 6), (100, 64)),
                            ((-1, 3, 5), (100, 64)), ((0, 4, 2), (100, 64)), ((0, 3, 2 ** 31 - 1), (100, 64)),
                            ((0, 3, 5), (-1, 64)), ((0, 3, 5), (size + 1, 64)), ((0, 3, 5), (2 ** 31 - 1, 64)),
                            ((0, 3, 5), (140 - n[0] + 1, 64))):  # (the last: a new token inside the prefix)
        fm.fm_attn_shared(q, s.cache, s.batch, fm.SharedPrefix(_i32(seq_off), _i32(prefix)), scale=0.125)
        assert fm.fm_device_status() == RANGE, (seq_off, prefix)
    for over in (dict(q_off=s.q_off + 1), dict(q_off=s.q_off.flip(0)), dict(kv_len=s.kv_len + 1000), dict(kv_len=-s.kv_len)):
        a = dict(q_off=s.q_off, kv_len=s.kv_len, page_table=s.table)
        a.update(over)
        fm.fm_attn_shared(q, s.cache, fm.PagedBatch(**a), s.shared, scale=0.125)
        assert fm.fm_device_status() == RANGE, list(over)
    for entry in (-1, s.cache.n_pages, 2 ** 31 - 1):
        for at in ((0, 0), (1, 6), (4, 4)):  # a shared page, pages of one sequence
            t = s.table.clone()
            t[at] = entry
            fm.fm_attn_shared(q, s.cache, fm.PagedBatch(s.q_off, s.kv_len, t), s.shared, scale=0.125)
            assert fm.fm_device_status() == RANGE, (entry, at)
    o2, l2 = fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=0.125)
    assert torch.equal(o, o2) and torch.equal(lse, l2) and fm.fm_device_status() == OK


def test_offsets_that_descend_plan_nothing_beyond_32_bits():
    # descending offsets: spans of all tokens, whose tiles times the CTAs pass 32 bits; nothing to attend to either
    R, Hkv, width = 9, 64, 1000
    cache = fm.fm_cache_new(1, Hkv, 128, 64)
    cache.k.zero_(), cache.v.fill_(1.0)
    kv_len = torch.full((R,), 128 * width, dtype=torch.int32).cuda()
    table = torch.zeros(R, width, dtype=torch.int32).cuda()
    q = torch.zeros(R, 16 * Hkv, 64, dtype=torch.bfloat16).cuda()
    shared = fm.SharedPrefix(_i32([0, 9, 9]), _i32([128 * 500, 0]))
    good = fm.PagedBatch(torch.arange(R + 1, dtype=torch.int32).cuda(), kv_len, table)
    for off, groups in ((_i32([0, R] * 5), shared), (good.q_off, fm.SharedPrefix(_i32([9, 0, 9]), _i32([0, 128 * 500])))):
        fm.fm_attn_shared(q, cache, fm.PagedBatch(off, kv_len, table), groups, scale=1.0)
        assert fm.fm_device_status() == RANGE
    o, lse = fm.fm_attn_shared(q, cache, good, shared, scale=1.0)
    assert (o == 1).all() and float((lse - torch.log(torch.tensor(128.0 * width))).abs().max()) <= 1e-5
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("Hq", [4, 32])
def test_graph_replay_with_other_lengths_and_groups(Hq, f8):
    s = Groups([400, 200], [[60, 70, 20], [90, 50]], [[1, 1, 1], [1, 1]], 2, 128, 16, f8, seed=81, Hq=Hq)
    q, o, lse = s.attend(Hq)
    q = q.cuda()
    o, lse = torch.empty_like(o), torch.empty_like(lse)
    ws = torch.empty(fm.fm_attn_shared_workspace_bytes(s.cache, s.batch, s.shared, 5, Hq), dtype=torch.uint8, device="cuda")

    def step():
        fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=128 ** -0.5, o=o, lse=lse, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for short, prefix, off in (((0, 0, 0, 0, 0), (400, 200), (0, 3, 5)), ((3, 60, 1, 9, 40), (390, 100), (0, 3, 5)),
                               ((0, 5, 0, 0, 0), (400, 0), (0, 2, 5)), ((10, 0, 19, 0, 0), (0, 200), (0, 3, 5))):
        keys = [a - b for a, b in zip(s.keys, short)]
        s.kv_len.copy_(torch.tensor(keys, dtype=torch.int32))
        s.prefix_len.copy_(torch.tensor(prefix, dtype=torch.int32))
        s.seq_off.copy_(torch.tensor(off, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        ws.fill_(0xff)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        k, v = ([(quantised(x[i].double())[0] if f8 else x[i].double()).transpose(0, 1)[:, :n] for x, n in zip(s.rows, keys)]
                for i in range(2))
        assert_paged(o, lse, paged(q.double().cpu(), k, v, s.q_off.tolist(), keys, 128 ** -0.5, True, 0, 0), 128)
    assert fm.fm_device_status() == OK


def test_two_calls_at_once():
    a = Groups([700, 90], [[40] * 6, [33] * 3], [[1] * 6, [1] * 3], 2, 128, 16, False, seed=82, Hq=32)
    b = Groups([300], [[50, 70, 90, 31]], [[20, 31, 33, 25]], 2, 64, 32, True, seed=83, Hq=8)
    qa, oa, la = a.attend(32)
    qb, ob, lb = b.attend(8)
    qa, qb, side = qa.cuda(), qb.cuda(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(5):
        o1, l1 = fm.fm_attn_shared(qa, a.cache, a.batch, a.shared, scale=128 ** -0.5)
        o2, l2 = fm.fm_attn_shared(qb, b.cache, b.batch, b.shared, scale=64 ** -0.5, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o1, oa) and torch.equal(l1, la) and torch.equal(o2, ob) and torch.equal(l2, lb)


def test_pages_far_into_a_large_cache():
    # the same pages at the end of a cache whose byte offsets pass 2^32
    for f8, new in ((False, [[1, 1, 1]]), (True, [[1, 1, 1]]), (False, [[20, 30, 25]]), (True, [[20, 30, 25]])):
        s = Groups([200], [[64, 30, 40]], new, 8, 128, 64, f8, seed=84, Hq=32)
        q, o, lse = s.attend(32)
        n, big = s.cache.n_pages, 70000
        c = fm.fm_cache_new(big, 8, 64, 128, dtype=s.cache.k.dtype)
        for x, y in ((c.k, s.cache.k), (c.v, s.cache.v), (c.k_exp, s.cache.k_exp), (c.v_exp, s.cache.v_exp)):
            if x is not None:
                x.view(torch.uint8)[big - n:] = y.view(torch.uint8)
        batch = fm.PagedBatch(s.q_off, s.kv_len, torch.where(s.table >= 0, s.table + (big - n), s.table))
        o2, l2 = fm.fm_attn_shared(q.cuda(), c, batch, s.shared, scale=128 ** -0.5)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
        assert fm.fm_device_status() == OK
        del c, s


def test_responses_to_one_question():
    # the whole path: a prompt appended, its responses forked from it (the partly filled page
    # copied for each), then token by token, all three operators in one captured step, against
    # one flashmask_attention over the packed question and responses
    Hq, Hkv, d, page, P, R, n = 8, 2, 128, 16, 90, 4, 7
    N = P + R * n
    g = torch.Generator().manual_seed(85)
    qkv = torch.randn(1, N, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    f, sc = fm.fm_rope_freqs(d, kind="yarn", factor=2.0, orig_len=64, device="cuda")
    wq, wk = (1 + 0.1 * torch.randn(2, d, generator=g)).cuda()
    pos = torch.cat([torch.arange(P)] + [torch.arange(P, P + n)] * R).int().cuda()
    # key j is seen by later rows of its response, prompt keys by all
    lts = torch.full((1, N), N, dtype=torch.int32)
    for r in range(R):
        lts[0, P + r * n:P + (r + 1) * n] = P + (r + 1) * n
    vec = [lts.cuda(), torch.full((1, N), N, dtype=torch.int32).cuda(), torch.zeros(1, N, dtype=torch.int32).cuda(),
           torch.zeros(1, N, dtype=torch.int32).cuda()]
    spec = fm.QKNormRope(positions=pos, inv_freq=f, rot_scale=sc, q_weight=wq, k_weight=wk)
    q, k, v = (t.transpose(1, 2) for t in qkv.split([Hq, Hkv, Hkv], 2))
    want = fm.flashmask_attention(q, k, v, *vec, causal=True, qk=spec)[0].transpose(0, 1)
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    w, left = P // page, P % page
    ids = torch.randperm(w + R * (1 + -(-(left + n) // page)), generator=g).int()
    cache = fm.fm_cache_new(ids.numel(), Hkv, page, d)
    width = -(-(P + n) // page)
    table = torch.full((R, width), -1, dtype=torch.int32)
    table[:, :w] = ids[:w]
    table[:, w:] = ids[w:w + R * (width - w)].view(R, -1)
    # (wide enough for the steps to share)
    table = torch.nn.functional.pad(table, (0, 500), value=-1).cuda()
    how = dict(inv_freq=f, rot_scale=sc, q_weight=wq, k_weight=wk)
    prompt = fm.PagedBatch(_i32([0, P]), _i32([P]), table[:1].contiguous())
    qp = fm.fm_cache_append(*qkv[0, :P].split([Hq, Hkv, Hkv], 1), cache, prompt, **how)
    o, _ = fm.fm_attn_paged(qp, cache, prompt, scale=d ** -0.5)
    # both sides round P and O once each: within 2^-7 twice
    assert rel(o, want[:P]) <= 2 * 2.0 ** -7
    fm.fm_cache_copy(cache, table[0, w].repeat(R - 1), table[1:, w].contiguous())
    kv_len = _i32([P] * R)
    batch = fm.PagedBatch(_off([1] * R), kv_len, table)
    shared = fm.SharedPrefix(_i32([0, R]), _i32([P]))
    assert (fm.fm_attn_shared_workspace_bytes(cache, batch, shared, R, Hq)
            > fm.fm_attn_paged_workspace_bytes(cache, batch, R, Hq))
    x = torch.zeros(R, Hq + 2 * Hkv, d, dtype=torch.bfloat16).cuda()
    qn, o, lse = torch.empty(R, Hq, d, dtype=torch.bfloat16).cuda(), torch.empty(R, Hq, d, dtype=torch.bfloat16).cuda(), torch.empty(R, Hq).cuda()
    ws = torch.empty(fm.fm_attn_shared_workspace_bytes(cache, batch, shared, R, Hq), dtype=torch.uint8, device="cuda")

    def step():
        kv_len.add_(1)
        fm.fm_cache_append(*x.split([Hq, Hkv, Hkv], 1), cache, batch, out=qn, **how)
        fm.fm_attn_shared(qn, cache, batch, shared, scale=d ** -0.5, o=o, lse=lse, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kv_len.fill_(P)
    rows = torch.arange(R) * n + P
    for i in range(n):
        x.copy_(qkv[0, rows + i])
        graph.replay()
        assert rel(o, want[rows + i]) <= 2 * 2.0 ** -7
        err = (o.double() - want[rows + i].double()).abs().max()
        assert float(err) <= 2 * 2.0 ** -7 * float(v.abs().max())
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("d, f8", [(128, False), (128, True), (64, False)])
def test_a_bound_of_the_prefixes_decides_whether_a_call_shares(d, f8):
    # a table with room for 32768 keys says nothing about prefixes of 100: sharing them loses (64 sequences of up
    # to 400 keys 36 us, for 24 apart)
    R, Hq, Hkv = 64, 32, 8
    s = Groups([100], [[1 + 7 * i % 300 for i in range(R)]], [[1] * R], Hkv, d, 64, f8, seed=91, pad=512)
    q, *shared = s.attend(Hq)
    q = q.cuda()
    apart = fm.fm_attn_paged(q, s.cache, s.batch, scale=d ** -0.5)
    assert not torch.equal(shared[0], apart[0])
    for most, want in ((100, apart), (63, apart), (30000, shared), (2 ** 30, shared), (0, shared)):
        s.shared = fm.SharedPrefix(s.seq_off, s.prefix_len, max_prefix=most)
        o, lse = fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=d ** -0.5)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), most
    # groups that are none are no error of a call that does not share
    s.shared = fm.SharedPrefix(s.seq_off + 1, s.prefix_len, max_prefix=100)
    fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=d ** -0.5)
    assert fm.fm_device_status() == OK


@pytest.mark.parametrize("d, f8", [(128, False), (64, True)])
def test_a_bound_of_the_prefixes_of_chunks(d, f8):
    new = [90, 70, 62, 64, 80, 50, 77, 67]
    s = Groups([1024], [new], [new], 4, d, 64, f8, seed=92, pad=512)
    for most, same in ((0, False), (1024, True)):
        s.shared = fm.SharedPrefix(s.seq_off, s.prefix_len, max_prefix=most)
        q, o, lse = s.attend(16)
        o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=d ** -0.5)
        assert (torch.equal(o, o2) and torch.equal(lse, l2)) == same


@pytest.mark.parametrize("P, R, n", [(3000, 8, 1), (3000, 40, 1), (6000, 16, 20)])
def test_prefixes_longer_than_their_bound(P, R, n):
    s = Groups([P], [[n + 5] * R], [[n] * R], 8, 128, 64, False, seed=93)
    for most, same in ((P - 100, False), (1, True)):
        s.shared = fm.SharedPrefix(s.seq_off, s.prefix_len, max_prefix=most)
        assert s.shared.max_prefix == most
        q, o, lse = s.attend(32)
        o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=128 ** -0.5)
        assert (torch.equal(o, o2) and torch.equal(lse, l2)) == same


@pytest.mark.parametrize("new, Hq", [([[1], [0, 1, 0], [1, 1]], 4), ([[1], [0, 1, 0], [1, 1]], 160),
                                     ([[20], [0, 33, 0], [25, 31]], 8), ([[1], [0, 3, 0], [2, 1]] + [[1]] * 260, 4)])
@pytest.mark.parametrize("f8", [False, True])
def test_a_prefix_that_one_sequence_alone_uses_is_no_prefix(new, Hq, f8):
    # a group of one, and one whose other sequences have no new tokens: as if the group's length were 0
    prefix = [300, 200, 90] + [37] * (len(new) - 3)
    s = Groups(prefix, [[40], [50, 60, 30], [30, 35]] + [[9]] * (len(new) - 3), new, 2, 64, 16, f8, seed=94, Hq=Hq)
    q, o, lse = s.attend(Hq)
    plain = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=0.125)
    s.prefix_len[0] = s.prefix_len[1] = 0
    s.prefix_len[3:] = 0
    o2, l2 = fm.fm_attn_shared(q.cuda(), s.cache, s.batch, s.shared, scale=0.125)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert not torch.equal(lse, plain[1])  # (the call shares)
    # lengths that no sequence has are flagged all the same
    s.prefix_len[0] = 340
    fm.fm_attn_shared(q.cuda(), s.cache, s.batch, s.shared, scale=0.125)
    assert fm.fm_device_status() == RANGE


@pytest.mark.parametrize("new, Hq", [([[0, 1, 1], [1, 0]], 8), ([[0, 1, 1], [1, 0]], 128), ([[0, 30, 20], [25, 0]], 8)])
def test_lengths_of_slots_out_of_use(new, Hq):
    # any that a length may be, without an effect; others are flagged, as those of slots in use, and nothing is written
    s = Groups([100, 64], [[40, 50, 60], [30, 35]], new, 2, 64, 16, False, seed=95, Hq=Hq)
    q, o, lse = s.attend(Hq)
    T, room = sum(s.new), 16 * s.table.shape[1]
    q, kv = q.cuda(), torch.randn(T, 4, 64, generator=s.g).to(torch.bfloat16).cuda()
    k, v = kv.split([2, 2], 1)
    fm.fm_cache_write(k, v, s.cache, s.batch)
    want = (fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=0.125), fm.fm_attn_paged(q, s.cache, s.batch, scale=0.125))
    held = [s.cache.k.clone(), s.cache.v.clone()]
    for length in (0, 1, room, -1, room + 1, 2 ** 31 - 1, -2 ** 31):
        bits = OK if 0 <= length <= room else RANGE
        for r in (0, 4):
            s.table[r] = -1 if r else 2 ** 30
            s.kv_len[r] = length
        got = fm.fm_attn_shared(q, s.cache, s.batch, s.shared, scale=0.125)
        assert fm.fm_device_status() == bits
        also = fm.fm_attn_paged(q, s.cache, s.batch, scale=0.125)
        assert fm.fm_device_status() == bits
        if bits == OK:
            assert all(torch.equal(a, b) for x, y in zip((got, also), want) for a, b in zip(x, y))
        for write in (lambda a, b: fm.fm_cache_write(a, b, s.cache, s.batch),
                      lambda a, b: fm.fm_cache_append(q, a, b, s.cache, s.batch)):
            for x, y in zip((s.cache.k, s.cache.v), held):
                x.copy_(y)
            write(-k, -v)
            assert fm.fm_device_status() == bits
            same = [torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip((s.cache.k, s.cache.v), held)]
            assert same == [bits == RANGE] * 2
        for x, y in zip((s.cache.k, s.cache.v), held):
            x.copy_(y)


@pytest.mark.parametrize("R, n, Hkv, P, pad, shares", [(32, 9, 4, 2000, 0, False), (32, 9, 4, 500, 2000, False),
                                                       (4, 18, 4, 3000, 0, False), (3, 8, 1, 2000, 0, True)])
@pytest.mark.parametrize("f8", [False, True])
def test_chunks_of_wide_heads_share_where_few_units_would_leave_the_rest_idle(R, n, Hkv, P, pad, shares, f8):
    # d = 256 has no kernel that reads a prefix for more than 16 rows: with as many units as CTAs sharing takes
    # up to 1.7 times as long (32 chunks of 30 tokens behind 8192 keys 2006 us, 1299 apart)
    s = Groups([P], [[n + 5] * R], [[n] * R], Hkv, 256, 64, f8, seed=96, pad=pad)
    q, o, lse = s.attend(4 * Hkv)
    o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=1 / 16)
    assert (torch.equal(o, o2) and torch.equal(lse, l2)) != shares


@pytest.mark.parametrize("new, Hq", [([[1, 1, 1], [1, 1]], 4), ([[1, 1, 1], [1, 1]], 128), ([[30, 20, 31], [25, 40]], 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [-120, -108, 100])
def test_quantised_values_far_from_one(new, Hq, d, power):
    # scales down to 2^-126 are further below a row's largest weight than exp2's smallest numbers
    # (such chunks at d = 256 are not shared)
    s = Groups([300, 140], [[40, 50, 60], [64, 45]], new, 2, d, 16, True, seed=97,
               Hq=None if d == 256 and new[0][0] > 1 else Hq)
    for x in s.rows:
        x[1] = (x[1].double() * 2.0 ** power).to(torch.bfloat16)
    s.write()
    q = torch.randn(sum(s.new), Hq, d, generator=s.g).to(torch.bfloat16)
    o, lse = fm.fm_attn_shared(q.cuda(), s.cache, s.batch, s.shared, scale=d ** -0.5)
    O, L, A, mag = s.reference(q, d ** -0.5, True)
    one = 2.0 ** -power  # (the bounds are relative)
    assert_paged(o.double() * one, lse, (O * one, L, A * one, mag), d)
    assert fm.fm_device_status() == OK
