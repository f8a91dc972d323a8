"""The range-checked debug library: the append, page copies and attention over shared
prefixes run clean under it, at parity with the 64-bit forms."""
import os
import subprocess
import sys

import pytest

from mask_aware_sparse_gb300 import build as fmbuild

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_build_shares_clean():
    fmbuild.build(debug=True)
    env = dict(os.environ, FM_LIBRARY="debug")
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_build_shared_case.py")], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "debug build clean" in r.stdout
