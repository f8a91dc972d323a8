"""GPU: chunk_kernel's rings of key tiles. Tiles of 128 keys hold rows that differ from those of the
next tiles in their bytes and scales, and each query looks at one tile alone, so that a row of
another tile, in a stage that was released or filled at the wrong time, shows.

Tile t's keys are 8 at column t % d and 0 elsewhere, a query 8 at its tile's column: scores are
28 in its tile, 0 elsewhere, where 2^14 keys weigh 2^14 / 128 e^-28 < 2^-33 of its tile's. A row of
another tile among the tile's keys takes 1 / 128 of the sum away: LSE moves by 2^-7; its bound is
2^-11. Columns are dealt to three classes in pieces of eight; tile t's values are s(t) = 8^(t % 3),
but 2^-6 s(t) in class -t % 3, where those of tiles u one, two and four places on are s(u). Eight
columns of such a tile, under a row's own scale, move that class by (64 - 1) / 128 of its value, a
whole row by (64 s(u) / s(t) - 1) / 128: 0.05 or more for two tiles of three at least. The bound is
2^-8 (O's rounding; equal weights' cancel) and 2^-9."""
import math

import pytest
import torch

import mask_aware_sparse_gb300 as fm

pytestmark = pytest.mark.gpu
OK = (fm.FM_OK, 0)
SCORE = 28


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _values(t, d):
    return torch.where((t[:, None] + torch.arange(d) // 8) % 3 == 0, 2.0 ** -6, 1.0) * (8.0 ** (t % 3))[:, None]


def _rows(tiles, Hkv, d):
    """Keys and values of the tiles, (128 tiles, Hkv, d), bf16."""
    t = torch.arange(tiles).repeat_interleave(128)
    k = torch.zeros(128 * tiles, d)
    k[torch.arange(128 * tiles), t % d] = 8.0
    v = _values(t, d)
    return [x.to(torch.bfloat16)[:, None].expand(-1, Hkv, -1).cuda() for x in (k, v)]


def _cache(rows, Hkv, d, page, f8, own=0):
    """A cache that holds the rows as one sequence's, pages shuffled, and `own` pages more; their numbers."""
    L = rows[0].shape[0]
    ids = torch.randperm(L // page + own, generator=torch.Generator().manual_seed(1)).int().cuda()
    cache = fm.fm_cache_new(ids.numel(), Hkv, page, d, dtype=torch.float8_e4m3fn if f8 else torch.bfloat16)
    for x in (cache.k, cache.v, cache.k_exp, cache.v_exp):
        if x is not None:
            x.view(torch.uint8).zero_()
    if f8:
        cache.k_exp.fill_(127), cache.v_exp.fill_(127)
    table = ids[:L // page][None].contiguous()
    fm.fm_cache_write(*rows, cache, fm.PagedBatch(_i32([0, L]), _i32([L]), table))
    assert fm.fm_device_status() == OK
    return cache, table, ids[L // page:]


def _check(o, lse, at, d):
    """Every query's O is its tile's values, its LSE that of 128 keys at 28."""
    want = _values(at, d)[:, None]
    err = ((o.double().cpu() - want) / want).abs()
    assert float(err.max()) <= 2.0 ** -8 + 2.0 ** -9, (int(err.amax((1, 2)).argmax()), float(err.max()))
    off = (lse.double().cpu() - (math.log(128) + SCORE)).abs()
    assert float(off.max()) <= 2.0 ** -11, (int(off.amax(1).argmax()), float(off.max()))


@pytest.mark.parametrize("d, tiles, G, page", [(128, 128, 4, 64), (128, 127, 8, 16), (64, 64, 4, 128), (64, 63, 2, 32)])
@pytest.mark.parametrize("f8", [False, True])
def test_tiles_of_one_sequence(d, tiles, G, page, f8):
    # a long chunk (cross attention): 13 key tiles a CTA and more, in two to four stages
    Hkv, T = 4, 2048 // G
    rows = _rows(tiles, Hkv, d)
    cache, table, _ = _cache(rows, Hkv, d, page, f8)
    at = (torch.arange(T) * 37 + 5) % tiles
    q = torch.zeros(T, Hkv * G, d)
    q[torch.arange(T), :, at % d] = 8.0
    batch = fm.PagedBatch(_i32([0, T]), _i32([128 * tiles]), table)
    for _ in range(4):
        o, lse = fm.fm_attn_paged(q.to(torch.bfloat16).cuda(), cache, batch, scale=SCORE / 64, causal=False)
        assert fm.fm_device_status() == OK
        _check(o, lse, at, d)


@pytest.mark.parametrize("d, tiles, G, page", [(128, 128, 8, 64), (128, 127, 4, 16), (64, 64, 8, 128), (64, 63, 8, 32)])
@pytest.mark.parametrize("n", [1, 9])
@pytest.mark.parametrize("f8", [False, True])
def test_tiles_of_a_shared_prefix(d, tiles, G, page, n, f8):
    # single tokens behind a prefix (chunk_kernel over it alone), and chunks
    Hkv, R = 4, 192 if n == 1 else 24
    T, L = R * n, 128 * tiles
    rows = _rows(tiles, Hkv, d)
    up = -(-n // page)
    cache, table, own = _cache(rows, Hkv, d, page, f8, R * up)
    table = torch.cat((table.expand(R, -1), own.view(R, up)), 1).contiguous()
    batch = fm.PagedBatch(_i32([n * r for r in range(R + 1)]), _i32([L + n] * R), table)
    shared = fm.SharedPrefix(_i32([0, R]), _i32([L]))
    at = (torch.arange(T) * 37 + 5) % tiles
    q = torch.zeros(T, Hkv * G, d)
    q[torch.arange(T), :, at % d] = 8.0
    q = q.to(torch.bfloat16).cuda()
    assert (fm.fm_attn_shared_workspace_bytes(cache, batch, shared, T, Hkv * G)
            > fm.fm_attn_paged_workspace_bytes(cache, batch, T, Hkv * G))
    plain = fm.fm_attn_paged(q, cache, batch, scale=SCORE / 64)
    for _ in range(4):
        o, lse = fm.fm_attn_shared(q, cache, batch, shared, scale=SCORE / 64)
        assert fm.fm_device_status() == OK
        _check(o, lse, at, d)
    _check(*plain, at, d)
