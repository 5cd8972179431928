"""Which kernel a paged decode call runs on: the choice follows the longest
unit's work as the window and the table bound it."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
import test_gpu_paged_decode as paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("lens,kernel", [((20011, 9), "paged_decode_mma"), ((300, 9), "paged_decode_cluster")],
                         ids=["long", "short"])
def test_a_window_past_every_length_changes_neither_kernel_nor_bits(D, lens, kernel):
    """Windows up to the largest that the call takes (a larger one is cut to it)."""
    scale = 1.0 / math.sqrt(D)
    q, k, v, table, nonpad = paged.make(lens, 4, 2, D, 16, torch.bfloat16)
    good = paged.run(q, k, v, table, nonpad, scale, 0)
    assert ek.extkv_last_kernel() == kernel
    for window in (lens[0], 1 << 30, 2 ** 31 - 33, 2 ** 31 - 16, 2 ** 31 - 1, 2 ** 31, 2 ** 40):
        y = paged.run(q, k, v, table, nonpad, scale, window)
        assert ek.extkv_last_kernel() == kernel, window
        assert torch.equal(y, good), window
