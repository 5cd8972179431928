"""The packed and paged operators on the library built with EXTKV_CHECKED
(device bounds checks that flag EXTKV_DEV_BOUNDS and skip the access): every
kernel, against the definition, with a clean status word.  Run as its own
process by tests/test_gpu_checked_paged.py, so that this library is the one
loaded; prints "checked ok <calls>" at the end."""
import math
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

import test_gpu_packed_prefill as prefill  # noqa: E402
import test_gpu_paged_decode as decode  # noqa: E402
import test_gpu_rotary_append as rotary  # noqa: E402
from packed_ref import check  # noqa: E402

B, F = torch.bfloat16, torch.float32
calls = 0
for lens, Hq, Hkv, D, page, window, dtype in [
        ((0, 1, 17, 257, 1000), 16, 8, 256, 16, 100, B), ((0, 1, 17, 257, 1000), 32, 2, 128, 64, 0, B),
        ((5000, 3), 8, 4, 64, 16, 0, B), ((5000, 3), 16, 2, 512, 32, 0, B), ((5000, 3), 6, 2, 128, 7, 0, B),
        ((0, 1, 17, 257), 4, 2, 96, 16, 0, B), ((0, 1, 17, 3000), 9, 1, 128, 24, 0, F)]:
    q, k, v, table, nonpad = decode.make(lens, Hq, Hkv, D, page, dtype, window=window)
    y = decode.run(q, k, v, table, nonpad, 1 / math.sqrt(D), window)
    ref, tol = decode.reference(q, k, v, table, lens, window, 1 / math.sqrt(D))
    check(y, ref, tol, f"decode {D}")
    calls += 1
for lens, Hq, Hkv, D, dtype, window in [((1, 0, 129, 300), 8, 4, 128, B, 0), ((1, 0, 129, 300), 6, 2, 64, B, 90),
                                        ((1, 0, 129, 300), 4, 2, 256, B, 0), ((1, 0, 129, 60), 4, 2, 96, B, 0),
                                        ((1, 0, 129, 60), 6, 2, 128, F, 20)]:
    q, k, v, cu = prefill.make(lens, Hq, Hkv, D, dtype, True, 3, 5)
    y = prefill.run(q, k, v, cu, 1 / math.sqrt(D), True, window)
    ref, tol = prefill.reference(q, k, v, cu, 1 / math.sqrt(D), True, window)
    check(y, ref, tol, f"prefill {D}")
    calls += 1
for case in rotary.APPEND:
    rotary.test_append_rotates_and_writes(case)
    calls += 1
print(f"checked ok {calls}")
