"""GPU: values at the edges of what the paged cache and its attention accept, and
calls that must be refused, against the 64-bit forms of serve_ref."""
import pytest
import torch

import mask_aware_sparse_gb300 as fm
from serve_ref import BF16_HALF, assert_paged, paged
from test_gpu_paged import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d, new", [(64, [1, 1, 1]), (64, [40, 30, 60]), (128, [40, 30, 60]), (256, [2, 1, 9])])
@pytest.mark.parametrize("byte", [0x7f, 0xff])
def test_nan_bytes_of_rows_with_an_ordinary_exponent(d, new, byte):
    # a cache that its owner filled by a plain conversion: e4m3's NaN, scales of numbers
    s = Setup([100, 90, 200], new, 2, d, 16, True, seed=30)
    q, o, lse = s.attend(4)
    at = (int(s.table[1, 0]), 1, 5, d // 2 + 3)  # key 5 of the second sequence, second head
    a, b = s.q_off.tolist()[1:3]
    others = torch.ones(o.shape[:2], dtype=torch.bool)
    others[a:b, 2:] = False
    for which in (0, 1):
        c = (s.cache.k, s.cache.v)[which].view(torch.uint8)
        was = c[at].clone()
        c[at] = byte
        o2, l2 = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=d ** -0.5)
        if which == 0:
            assert torch.isnan(l2[a:b, 2:]).all() and torch.isnan(o2[a:b, 2:]).all()
        else:
            assert torch.isnan(o2[a:b, 2:, at[3]]).all() and torch.equal(l2, lse)
        assert torch.equal(o2[others.cuda()], o[others.cuda()]) and torch.equal(l2[others.cuda()], lse[others.cuda()])
        got = fm.fm_cache_read(s.cache, s.kv_off, s.table, 390)[which][0]
        hit = torch.zeros(got.shape, dtype=torch.bool)
        hit[1, 105, at[3]] = True
        assert torch.equal(torch.isnan(got).cpu(), hit)
        c[at] = was
    assert fm.fm_device_status() == (fm.FM_OK, 0)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


RANGE = (fm.FM_ERR_DEVICE, fm.FM_DEVERR_RANGE)


@pytest.mark.parametrize("off", [(0, 6, 5), (0, 3, 9), (3, 1, 5), (-4, 3, 5), (2, 3, 5), (0, 3, 2 ** 31 - 1),
                                 (0, -1, 5), (5, 0, 0)])
@pytest.mark.parametrize("f8", [False, True])
def test_cache_calls_flag_offsets_and_write_nothing(off, f8):
    cache = fm.fm_cache_new(4, 2, 16, 64, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16)
    table, kv_len = _i32(0, 1, 2, 3).view(2, 2), _i32(20, 5)
    held = torch.randn(2, 52, 2, 64, generator=torch.Generator().manual_seed(31)).to(torch.bfloat16).cuda()
    fm.fm_cache_write(held[0], held[1], cache, fm.PagedBatch(_i32(0, 32, 52), _i32(32, 20), table))
    state = [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp) if t is not None]
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16).cuda()
    assert fm.fm_device_status() == (fm.FM_OK, 0)
    fm.fm_cache_write(x, x, cache, fm.PagedBatch(_i32(*off), kv_len, table))
    assert fm.fm_device_status() == RANGE
    now = [t.view(torch.uint8) for t in (cache.k, cache.v, cache.k_exp, cache.v_exp) if t is not None]
    assert all(torch.equal(a, b) for a, b in zip(state, now))
    fm.fm_cache_read(cache, _i32(*off), table, 5)
    assert fm.fm_device_status() == RANGE


@pytest.mark.parametrize("kv_len, new", [((33, 5), (0, 2, 5)), ((-1, 5), (0, 0, 3)), ((20, 2 ** 31 - 1), (0, 2, 2)),
                                         ((-(2 ** 31), 5), (0, 2, 5))])
def test_a_write_flags_lengths_and_writes_nothing(kv_len, new):
    cache = fm.fm_cache_new(4, 2, 16, 64)
    cache.k.zero_(), cache.v.zero_()
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16).cuda()
    fm.fm_cache_write(x, x, cache, fm.PagedBatch(_i32(*new), _i32(*kv_len), _i32(0, 1, 2, 3).view(2, 2)))
    assert fm.fm_device_status() == RANGE
    assert not cache.k.any() and not cache.v.any()


def test_offsets_of_many_sequences_are_looked_at():
    # more than a block has threads; one pair of offsets descends where no token of most blocks is
    R = 1000
    cache = fm.fm_cache_new(R, 1, 16, 64)
    cache.k.zero_(), cache.v.zero_()
    off = torch.arange(R + 1, dtype=torch.int32)
    kv_len, table = torch.ones(R, dtype=torch.int32).cuda(), torch.arange(R, dtype=torch.int32)[:, None].contiguous().cuda()
    x = torch.ones(R, 1, 64, dtype=torch.bfloat16).cuda()
    bad = off.clone()
    bad[700], bad[701] = 701, 700
    fm.fm_cache_write(x, x, cache, fm.PagedBatch(bad.cuda(), kv_len, table))
    assert fm.fm_device_status() == RANGE
    assert not cache.k.any() and not cache.v.any()
    fm.fm_cache_write(x, x, cache, fm.PagedBatch(off.cuda(), kv_len, table))
    assert fm.fm_device_status() == (fm.FM_OK, 0)
    assert (cache.k[:, 0, 0] == 1).all() and not cache.k[:, 0, 1:].any()


@pytest.mark.parametrize("new, keys", [([3, 2], [20, 5]), ([300, 200], [700, 300]), ([1] * 300, [20] * 300)])
def test_attention_flags_offsets_that_do_not_start_at_0(new, keys):
    # planned by every CTA (whole units, divided ones) and by a kernel of its own
    s = Setup(keys, new, 2, 64, 16, False, seed=32)
    q = torch.ones(sum(new) + 1, 4, 64, dtype=torch.bfloat16).cuda()
    fm.fm_attn_paged(q, s.cache, s.batch, scale=0.1)
    assert fm.fm_device_status() == (fm.FM_OK, 0)
    fm.fm_attn_paged(q, s.cache, fm.PagedBatch(s.q_off + 1, s.kv_len, s.table), scale=0.1)
    assert fm.fm_device_status() == RANGE


@pytest.mark.parametrize("d, Hq", [(64, 4), (128, 32), (256, 4)])
@pytest.mark.parametrize("power, scale", [(-112, 0.125), (-100, 0.125), (112, 0.125), (0, 1e-30)])
def test_steps_over_quantised_keys_far_from_one(d, Hq, power, scale):
    # scores near 1 from queries near 2^power and keys near 2^-power; a scale so small that all weights are alike
    s = Setup([150, 33], [1, 1], 2, d, 16, True, seed=33)
    s.k = (s.k.double() * 2.0 ** -power).to(torch.bfloat16)
    fm.fm_cache_write(s.k.cuda(), s.v.cuda(), s.cache, fm.PagedBatch(s.kv_off, s.kv_len, s.table))
    q = (torch.randn(2, Hq, d, generator=s.g).double() * 2.0 ** power).to(torch.bfloat16)
    o, lse = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=scale)
    k, v = s.values()
    assert_paged(o, lse, paged(q.double(), k, v, s.q_off.tolist(), s.keys, scale, True, 0, 0), d)


@pytest.mark.parametrize("scale", [0.125, 1e-9, 1e-30])
def test_queries_of_zero_over_quantised_keys(scale):
    s = Setup([150, 33], [1, 1], 2, 64, 16, True, seed=34)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    q[1, 2] = 1.0
    o, lse = fm.fm_attn_paged(q.cuda(), s.cache, s.batch, scale=scale)
    k, v = s.values()
    assert_paged(o, lse, paged(q.double(), k, v, s.q_off.tolist(), s.keys, scale, True, 0, 0), 64)


@pytest.mark.parametrize("d, Hq", [(64, 2), (128, 32), (256, 4)])
@pytest.mark.parametrize("keys", [30, 500])
def test_quantised_values_of_rows_with_far_scales(d, Hq, keys):
    # a row 2^20 times the others' size, zero in some columns: there the others' values count
    s = Setup([keys, 20], [1, 1], 2, d, 16, True, seed=35)
    v = s.v.clone()
    v[3] = v[3] * 2.0 ** 20
    v[3, :, ::3] = 0
    s.v = v
    fm.fm_cache_write(s.k.cuda(), s.v.cuda(), s.cache, fm.PagedBatch(s.kv_off, s.kv_len, s.table))
    s.attend(Hq)


def _two_pi(bits):
    """2 pi * 2^bits by Machin's formula, in whole numbers."""
    def arctan(n):  # arctan(1 / n)
        t = s = (1 << bits + 32) // n
        k = 1
        while t:
            t, k = t // (n * n), k + 2
            s += t // k if k % 4 == 1 else -(t // k)
        return s
    return 8 * (4 * arctan(5) - arctan(239)) >> 32


@pytest.mark.parametrize("inter", [False, True])
def test_angles_at_far_positions_of_any_frequency(inter):
    # theta = pos * f exactly, modulo a turn: neither the product nor 1 / (2 pi) has enough of 64 bits
    f = torch.tensor([1.0, 0.7, 50.0, 1000.0, 1e6, 4e9, 1e-6, -1.0, -0.3, -1e5, 2.0 ** -40, 0.0, 1e-42, 16777217.0,
                      2.0 ** 24, 3.0], dtype=torch.float32)
    pos = torch.tensor([0, 1, -1, 12345, 2 ** 24 + 1, 2 ** 31 - 1, -(2 ** 31), 999999937], dtype=torch.int32)
    turn = _two_pi(200)
    theta = torch.empty(len(pos), len(f), dtype=torch.float64)
    for i, p in enumerate(pos.tolist()):
        for j, x in enumerate(f.tolist()):
            num, den = x.as_integer_ratio()
            theta[i, j] = ((p * num << 200) // den % turn) / (1 << 200)
    c, s = torch.cos(theta), torch.sin(theta)
    q = torch.ones(1, 1, len(pos), 64, dtype=torch.bfloat16).cuda()
    out = fm.fm_qk_norm_rope(q, q.clone(), positions=pos.cuda(), inv_freq=f.cuda(), interleaved=inter)[0]
    got = out[0, 0].double().cpu()
    a, b = (got[:, 0:32:2], got[:, 1:32:2]) if inter else (got[:, :16], got[:, 16:32])
    for x, want in ((a, c - s), (b, c + s)):
        # theta's rounding to fp32 (2^-24 of half a turn), cos and sin (2^-22), one bf16 rounding
        assert bool(((x - want).abs() <= BF16_HALF * want.abs() * 1.01 + 2.0 ** -20).all())
    assert (got[:, 32:] == 1).all()
