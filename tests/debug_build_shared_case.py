"""Run by tests/test_gpu_debug_shared.py in a fresh process with FM_LIBRARY=debug: the
append, page copies and attention over shared prefixes in the range-checked debug library
on small cases, checked against the 64-bit forms; exits non-zero on a parity failure or any
device error bit."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import mask_aware_sparse_gb300 as fm  # noqa: E402
from test_gpu_append import CASES, test_append_is_norm_rotation_and_write, test_copy  # noqa: E402
from test_gpu_shared import Groups, ones  # noqa: E402


def main():
    assert fm.LIB_PATH.endswith("libfm_debug.so"), fm.LIB_PATH
    for f8 in (False, True):
        for case in CASES[:6]:
            test_append_is_norm_rotation_and_write(case, f8)
        test_copy(3, 128, 32, f8, 7)
        for d in (64, 128, 256):
            # few rows, both kernels, one kernel for all, planned by a kernel of its own
            for prefix, rest, new, Hq, Hkv, page in (
                    ([300, 40], [[20, 3], [50, 9, 1]], None, 4, 2, 16), ([500], [[33] * 20], None, 8, 1, 64),
                    ([700, 64], [[60, 70, 35], [90, 40]], [[20, 31, 33], [25, 40]], 8, 2, 32),
                    ([100], [[9] * 60], [[5, 9] * 30], 4, 2, 128)):
                s = Groups(prefix, rest, new or ones(rest), Hkv, d, page, f8, seed=90, Hq=Hq)
                s.attend(Hq)  # (asserts that no error bit is set)
                s.attend(Hq, causal=False)
    st, bits = fm.fm_device_status()
    if st != fm.FM_OK:
        raise SystemExit(f"device status {st} bits {bits}")
    print("debug build clean")


if __name__ == "__main__":
    main()
