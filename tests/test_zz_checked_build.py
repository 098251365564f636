"""The bounds-checked build (libinfllmv2_checks.so: device index checks that
set INFLLMV2_STATUS_CHECK and skip the access, in place of a memory
sanitizer) runs the smoke prefill and decode step against the oracle with no
check failing.  A separate process, since a process loads one build."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_checked_build_runs_clean(cuda_lib):
    from trainable_block_sparse_compressed_b200 import build
    lib = build.build(checks=True)
    env = dict(os.environ, INFLLMV2_LIB=lib)
    r = subprocess.run([sys.executable, "-c", "import __graft_entry__ as g; g.smoke()"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert "smoke ok" in r.stdout


def test_window_and_pages_run_clean_on_the_checked_build(cuda_lib):
    """The tests of the windowed attention, its gradients and the paged cache
    that assert an empty status, on the checked build."""
    from trainable_block_sparse_compressed_b200 import build
    lib = build.build(checks=True)
    tests = [os.path.join(ROOT, "tests", f"test_{x}.py")
             for x in ("paged", "window_attn", "window_attn_backward")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider", "-k",
                        "all_elements or serving or split or short_windows or tables or past", *tests],
                       cwd=ROOT, env=dict(os.environ, INFLLMV2_LIB=lib), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
