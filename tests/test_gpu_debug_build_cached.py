"""The bounds-checked FA_DEBUG build on the norm, rotation, append and 4-bit
decode kernels: on valid inputs no check fires and the results are the release
build's bit for bit. The debug library runs in a child process."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_build_matches_release_bitwise(tmp_path):
    from exact_tiled_attention_24_gb300 import build
    build.build()
    build.build(debug=True)
    import cached_debug_cases
    import exact_tiled_attention_24_gb300 as fa
    assert not fa.debug_checks()
    release = cached_debug_cases.run_cases()
    path = tmp_path / "debug.pt"
    r = subprocess.run([sys.executable, os.path.join(HERE, "cached_debug_cases.py"), str(path)],
                       env=dict(os.environ, FA_DEBUG_LIBRARY="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    debug = torch.load(path)
    assert sorted(debug) == sorted(release)
    for name, t in release.items():
        assert torch.equal(t, debug[name]), name
