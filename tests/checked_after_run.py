"""The shared prefix with own slots after it, on the library built with EXTKV_CHECKED: results
against the definition, no access outside its buffer, and the kinds of buffers that the
kernels address by computed indexes all tested (status[3]).  Run as its own process by
tests/test_gpu_own_slots_after.py; prints "checked ok <calls>" at the end."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import torch  # noqa: E402

from biased_gqa_attention_gb300 import build  # noqa: E402
from biased_gqa_attention_gb300 import extkv as ek  # noqa: E402

lib = ek.load(build.build(checked=True))
assert os.path.basename(lib._name) == "libextkv_checked.so", lib._name

from packed_ref import check  # noqa: E402
from test_gpu_own_slots_after import AFTER, lens, wide  # noqa: E402
from test_gpu_shared_prefix import make, reference, run  # noqa: E402

LENS, TABLE, ROWS, PAGES, OUT, PARTIAL = (1 << i for i in range(6))  # common.cuh
calls = 0
for prefix, sizes, Hq, Hkv, page, window in [
        ((700,), (90,), 8, 2, 16, 0), ((700, 33), (90, 1), 8, 2, 64, 300), ((700,), (90,), 6, 2, 48, 0)]:
    s = wide(make(prefix, sizes, lens(sum(sizes) + 1), Hq, Hkv, 128, page, torch.bfloat16, window=window))
    st = ek.new_status()
    y = run(s, 0.1, window, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK, ek.extkv_last_error()
    assert ek.extkv_last_kernel() == AFTER
    tested = int(st[3])  # (own pages by requests: no index to test)
    assert tested == LENS | TABLE | ROWS | OUT | PARTIAL, f"{tested:#x}"
    ref, tol = reference(s, 0.1, window)
    check(y, ref, tol, "y")
    calls += 1
print(f"checked ok {calls}")
