"""Wide tables, single entries and rotary widths on the bounds-checked build, in
a child process that loads it."""
import pytest

from test_gpu_checked import _run_child

pytestmark = pytest.mark.gpu


def test_kv_wide_suites_run_clean_on_the_checked_build():
    r = _run_child(["-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_kv_evict_wide.py",
                    "tests/test_gpu_kv_attn_places.py", "tests/test_gpu_norm_rope_unrotated.py"], timeout=900)
    assert r.returncode == 0, r.stdout[-4000:]
