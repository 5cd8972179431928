"""The packed and paged operators on the library built with EXTKV_CHECKED, in a
process of its own: results against the definition, clean status words."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_checked_build_runs_the_packed_and_paged_operators_without_a_bounds_flag():
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_paged_run.py")], capture_output=True, text=True,
                       timeout=1800, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "checked ok" in r.stdout, r.stdout[-2000:]
