"""What the kernels of attention over shared prefixes and of the append do in an order that
a GPU test sees only by chance, read from their source."""
import re

from test_serve_source import _kernels


def test_staged_tiles_are_released_after_a_fence():
    # reads of a staged e4m3 tile, then the copy that overwrites it: an arrival alone orders neither
    # loads on their way nor the two proxies
    body = dict(_kernels())["chunk_kernel"]
    release = body.index("mbar_arrive(&bars[C::REMPTY + rs])")
    loads = body.rindex("lds128(src", 0, release)
    between = re.sub(r"\s+", " ", body[loads:release])
    assert re.search(r"fence_proxy_async_smem\(\); __syncwarp\(\); if \(lane == 0\) $", between), between


def test_new_kernels_are_found():
    assert {"append_kernel", "copy_kernel", "merge_kernel"} <= {n for n, _ in _kernels()}
