"""GPU: forms of the attention over the paged cache beside one another: windows over
quantised caches of every head dim, prompts of d = 256, batches of chunks and single
tokens, calls of several streams in one captured graph; against the 64-bit forms."""
import pytest
import torch

import mask_aware_sparse_gb300 as fm
from test_gpu_paged import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window, sinks", [(1, 0), (64, 3), (100, 70), (1000, 4)])
@pytest.mark.parametrize("new, keys, d", [([1, 1], [900, 20], 64), ([1, 1], [900, 20], 128), ([1, 1], [900, 20], 256),
                                          ([70, 3], [500, 300], 64), ([300], [700], 128), ([40, 130], [600, 131], 128),
                                          ([30, 9], [500, 60], 256)])
@pytest.mark.parametrize("page", [16, 128])
def test_windows_over_quantised_caches(window, sinks, new, keys, d, page):
    s = Setup(keys, new, 2, d, page, True, seed=50)
    s.attend(8, window=window, sinks=sinks)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("new, keys, Hq, Hkv", [([500], [500], 4, 2), ([200], [1500], 8, 1), ([130, 1, 0, 77], [130, 600, 40, 300], 6, 2)])
@pytest.mark.parametrize("window", [0, 90])
def test_chunks_of_head_dim_256(f8, new, keys, Hq, Hkv, window):
    s = Setup(keys, new, Hkv, 256, 64, f8, seed=51)
    s.attend(Hq, window=window, sinks=4 if window else 0)
    if not window:
        s.attend(Hq, causal=False)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("chunk, singles", [(300, 63), (900, 64), (40, 10), (500, 200)])
def test_a_chunk_beside_single_tokens(f8, d, chunk, singles):
    # few rows a sequence on average, or many: one kernel takes them all either way
    g = torch.Generator().manual_seed(52)
    keys = torch.randint(1, 400, (singles,), generator=g).tolist()
    at = singles // 2
    s = Setup(keys[:at] + [chunk + 150] + keys[at:], [1] * at + [chunk] + [1] * (singles - at), 2, d, 32, f8, seed=53)
    s.attend(4)
    s.attend(4, window=60, sinks=2)


def test_calls_of_two_streams_in_one_graph():
    # a captured step that forks: each branch starts with a launch behind an event of the other
    # stream, both read what one write left, and the norm runs on what a copy filled
    a = Setup([700, 90], [1, 1], 2, 128, 16, False, seed=54)
    qkv = torch.randn(1, 2, 12, 128, generator=a.g).to(torch.bfloat16).cuda()
    stage = torch.zeros_like(qkv)
    f, _ = fm.fm_rope_freqs(128, device="cuda")
    pos = torch.tensor([699, 89], dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    outs = [[torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, device="cuda")] for _ in range(2)]
    ws = [torch.empty(fm.fm_attn_paged_workspace_bytes(a.cache, a.batch, 2, 8), dtype=torch.uint8, device="cuda")
          for _ in range(2)]

    def step():
        stage.copy_(qkv)
        q, k, v = (t.transpose(1, 2) for t in stage.split([8, 2, 2], 2))
        fm.fm_qk_norm_rope(q, k, positions=pos, inv_freq=f, out=(q, k))
        fm.fm_cache_write(stage[0, :, 8:10], stage[0, :, 10:], a.cache, a.batch)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        fm.fm_attn_paged(stage[0, :, :8], a.cache, a.batch, scale=0.1, o=outs[1][0], lse=outs[1][1], ws=ws[1], window=50,
                         stream=side)
        fm.fm_attn_paged(stage[0, :, :8], a.cache, a.batch, scale=0.1, o=outs[0][0], lse=outs[0][1], ws=ws[0])
        here.wait_stream(side)
        outs[0][0].add_(outs[1][0])  # both branches done

    main = torch.cuda.Stream()
    with torch.cuda.stream(main):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            step()
    for i in range(20):
        qkv.copy_(torch.randn(qkv.shape, generator=a.g).to(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for pair in outs for t in pair]
        with torch.cuda.stream(main):
            step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, [t for pair in outs for t in pair]))
    assert fm.fm_device_status() == (fm.FM_OK, 0)
