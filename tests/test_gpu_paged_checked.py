"""The paged-cache suite again under the checked build (libjamba_checked.so), whose device
checks of page numbers, lengths and slots must not fire on valid inputs (the conftest reads the
status word after every test there)."""
import os
import subprocess
import sys

import pytest

from tests.helpers import cuda_or_skip

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(os.environ.get("JAMBA_CHECKED", "0") == "1", reason="starts the checked build; not again inside it")
def test_paged_suite_under_the_checked_build():
    cuda_or_skip()
    from mamba_selective_scan_mixer_b200 import build
    if not os.path.exists(build.LIB_CHECKED):
        pytest.fail("libjamba_checked.so is not built (python -m mamba_selective_scan_mixer_b200.build --checked)")
    env = dict(os.environ, JAMBA_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_paged.py", "-m", "gpu", "-q", "-x",
                        "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
