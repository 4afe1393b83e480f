"""The host code of the norm's, the paged caches' and the drafted tokens' entry points
(argument checks, plans, workspace sizes) under AddressSanitizer, on the CPU: their ABI
tests run in a child process against the instrumented build of the library."""
import os
import subprocess
import sys

import pytest

from sparse_attention_indexer_block_amd.build import asan_runtime, build_host_asan
from test_host_asan import HERE, ROOT
from test_host_asan_attention import RUNNER


@pytest.mark.slow
def test_paged_abi_under_host_asan(tmp_path):
    rt = asan_runtime()
    if not rt:
        pytest.skip("the toolchain has no AddressSanitizer runtime")
    lib = build_host_asan(str(tmp_path))
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt + (os.pathsep + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:exitcode=86"
    env["PYTHONPATH"] = os.pathsep.join(p for p in (ROOT, HERE, env.get("PYTHONPATH", "")) if p)
    r = subprocess.run([sys.executable, "-c", RUNNER, lib, os.path.join(HERE, "test_abi_paged.py")], env=env, capture_output=True,
                       text=True, timeout=900, cwd=ROOT)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]
