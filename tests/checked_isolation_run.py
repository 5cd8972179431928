"""The shared prefix with windows and an infinity in its pages, on the library built with
EXTKV_CHECKED: results against the definition, no access outside its buffer, and q and the pools
tested where rows are attended alone (status[3]).  Run as its own process by
tests/test_gpu_window_isolation.py; prints "checked ok <calls>" at the end."""
import math
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

from biased_gqa_attention_gb300 import build  # noqa: E402
from biased_gqa_attention_gb300 import extkv as ek  # noqa: E402

lib = ek.load(build.build(checked=True))
assert os.path.basename(lib._name) == "libextkv_checked.so", lib._name

from test_gpu_shared_prefix import make, reference, run  # noqa: E402
from test_gpu_window_isolation import CASES, expect, poison  # noqa: E402

ROWS, PAGES = 0x4, 0x8  # common.cuh
calls = 0
for prefix, sizes, lens, Hq, Hkv, D, page, window, dtype in CASES:
    s = make(prefix, sizes, lens, Hq, Hkv, D, page, dtype, window=window)
    ref, tol = reference(s, 0.1, window)
    hit = poison(s, [("v", 0, prefix[0] - window + 70, Hkv - 1, 5, math.inf)])
    st = ek.new_status()
    y = run(s, 0.1, window, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK, ek.extkv_last_error()
    assert int(st[3]) & (ROWS | PAGES) == ROWS | PAGES, hex(int(st[3]))
    expect(s, y, ref, tol, hit, window)
    calls += 1
print(f"checked ok {calls}")
