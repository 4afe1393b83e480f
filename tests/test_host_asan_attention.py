"""The host code of the caches' and the attention's entry points (argument checks,
the plan of a call, workspace sizes) under AddressSanitizer, on the CPU: their ABI
tests run in a child process against the instrumented build of the library."""
import os
import subprocess
import sys

import pytest

from sparse_attention_indexer_block_amd.build import asan_runtime, build_host_asan
from test_host_asan import HERE, ROOT

RUNNER = r"""
import sys
import sparse_attention_indexer_block_amd as S
S.LIB_PATH = sys.argv[1]
import pytest
sys.exit(pytest.main(["-q", "-m", "not gpu", "-p", "no:cacheprovider", *sys.argv[2:]]))
"""


@pytest.mark.slow
def test_attention_abi_under_host_asan(tmp_path):
    rt = asan_runtime()
    if not rt:
        pytest.skip("the toolchain has no AddressSanitizer runtime")
    lib = build_host_asan(str(tmp_path))
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt + (os.pathsep + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:exitcode=86"
    env["PYTHONPATH"] = os.pathsep.join(p for p in (ROOT, HERE, env.get("PYTHONPATH", "")) if p)
    tests = [os.path.join(HERE, t) for t in ("test_abi_attention.py", "test_abi_attention_limits.py")]
    r = subprocess.run([sys.executable, "-c", RUNNER, lib, *tests], env=env, capture_output=True, text=True, timeout=900, cwd=ROOT)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]
