"""GPU: values at the edges of what the paged cache and its attention accept, and
calls that must be refused, against the 64-bit forms of serve_ref."""
import pytest
import torch

import mask_aware_sparse_gb300 as fm
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
