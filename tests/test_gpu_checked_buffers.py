"""The packed and paged operators on the library built with EXTKV_CHECKED, in a
process of its own: clean status words, and every kind of buffer tested that a
call addresses by computed indexes."""
import os
import re
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.gpu
def test_every_kind_of_buffer_is_tested_and_no_access_leaves_one():
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_buffers_run.py")], capture_output=True, text=True,
                       timeout=1800, cwd=ROOT)
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "checked ok" in r.stdout, r.stdout[-2000:]


def test_the_run_knows_the_kinds_of_the_source():
    """The values that the run expects in status[3] are the source's."""
    text = open(os.path.join(ROOT, "biased_gqa_attention_gb300", "csrc", "common.cuh")).read()
    kinds = re.findall(r"kChk(\w+) = (0x[0-9a-f]+)", text)
    assert [int(v, 16) for _, v in kinds] == [1 << i for i in range(8)]
    run = open(os.path.join(HERE, "checked_buffers_run.py")).read()
    names = re.search(r"^(.*) = \(1 << i for i in range\(8\)\)", run, re.M).group(1).split(", ")
    assert [n.lower() for n in names] == [k.lower() for k, _ in kinds]
