"""The decode over 8-bit pages where queries are near the least normal numbers or below, and the scale
makes up for it: brought into fp16's range, they keep their bits."""
import pytest
import torch

import test_gpu_fp8_pages as fp8
from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("algo", [ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO], ids=["axis", "auto"])
@pytest.mark.parametrize("power", [-90, -101, -113, -124, -132])
@pytest.mark.parametrize("D,page,dtype", [(64, 16, F32), (128, 16, F32), (256, 32, F32), (48, 16, F32), (128, 16, BF), (512, 16, BF)],
                         ids=lambda x: str(x))
def test_tiny_queries(D, page, dtype, power, algo):
    lens = (300, 40)
    q, k, v, sc, table, nonpad = fp8.make(lens, 4, 2, D, page, dtype, sigma=1.0)
    q = (q.double() * 2.0 ** power).to(dtype)
    q[1, 0] = 0.0
    assert 0 < float(q[0].abs().max()) < 2.0 ** (power + 4)
    scale = 2.0 ** min(-power - 3, 127)
    with ek.use_algo(algo):
        y = fp8.run(q, k, v, sc, table, nonpad, scale, 0)
    ref, tol = fp8.reference(q, k, v, sc, table, lens, 0, scale)
    check(y, ref, tol, "y")
