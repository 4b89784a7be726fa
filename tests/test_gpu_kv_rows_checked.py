"""The operators on the paged cache in the context's type on the bounds-checked
build: their tests run again in a child process that loads it; a store outside
its buffer is skipped and reported through the error word, which the tests find
clean."""
import pytest

from test_gpu_checked import _run_child

pytestmark = pytest.mark.gpu


def test_kv_rows_suite_runs_clean_on_the_checked_build():
    r = _run_child(["-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_kv_rows.py",
                    "tests/test_gpu_kv_rows_together.py"], timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:]
