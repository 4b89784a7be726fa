"""The verifier's side and the draft on an 8-bit cache on the bounds-checked
build: tests/test_gpu_verifier.py and tests/test_gpu_draft_kv8.py run again in
a child process that loads it.  Every output store of those
kernels is then compared with its buffer's extent; one outside is skipped and
reported through the error word, which the tests find clean."""
import pytest

from test_gpu_checked import _run_child

pytestmark = pytest.mark.gpu


def test_verifier_suite_runs_clean_on_the_checked_build():
    r = _run_child(["-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_verifier.py",
                    "tests/test_gpu_draft_kv8.py"],
                   timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:]
