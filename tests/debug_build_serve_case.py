"""Run by tests/test_gpu_debug_serve.py in a fresh process with FM_LIBRARY=debug: the
kernels of the norm and rotation, the paged cache and its attention in the
range-checked debug library on small cases, checked against the 64-bit forms; exits
non-zero on a parity failure or any device error bit."""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import mask_aware_sparse_gb300 as fm  # noqa: E402
from test_gpu_paged import Setup  # noqa: E402
from test_gpu_qk import CASES, test_forward_and_backward  # noqa: E402


def main():
    assert fm.LIB_PATH.endswith("libfm_debug.so"), fm.LIB_PATH
    for case in CASES[:6]:
        test_forward_and_backward(case, True)
    for f8 in (False, True):
        for d in (64, 128, 256):
            # single tokens, chunks of one and two query tiles, divided and whole units, sequences' ends
            for keys, new, Hq, Hkv, page in (([100, 1, 0, 700], [1, 1, 0, 1], 4, 2, 16), ([300], [300], 4, 2, 64),
                                             ([1500, 70], [40, 70], 8, 1, 32), ([20] * 40, [20] * 40, 2, 2, 128)):
                s = Setup(keys, new, Hkv, d, page, f8, seed=40)
                s.attend(Hq)  # (asserts that no error bit is set)
                s.attend(Hq, window=33, sinks=5)
            k, v = fm.fm_cache_read(s.cache, s.kv_off, s.table, sum(s.keys))
    st, bits = fm.fm_device_status()
    if st != fm.FM_OK:
        raise SystemExit(f"device status {st} bits {bits}")
    print("debug build clean")


if __name__ == "__main__":
    main()
