"""Which kernel a paged decode call runs on (the choice follows the longest unit's
work as the window and the table bound it), and the rows of a chunk as sequences
that share pages."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
import packed_ref
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


@pytest.mark.parametrize("width", [9, 152, 512, 4096])
def test_a_wide_table_changes_the_kernel_at_most(width):
    """The same sequence in tables of other widths: the definition's result, on whichever kernel."""
    q, k, v, table, nonpad = paged.make((130,), 16, 8, 256, 16, torch.bfloat16)
    wide = torch.full((1, width), -1, dtype=torch.int64, device="cuda")
    wide[:, :9] = table[:, :9]
    y = paged.run(q, k, v, wide, nonpad, 0.06, 0)
    # a unit's bytes on one of 8 CTAs against an equal share of 8 units: 180e3 bytes more at most
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    short = width * 16 * 256 * 4 * (1 / 8 - 8 / sms) <= 180e3  # 2428 slots with 152 SMs
    assert ek.extkv_last_kernel() == ("paged_decode_cluster" if short else "paged_decode_mma")
    ref, tol = paged.reference(q, k, v, wide, (130,), 0, 0.06)
    packed_ref.check(y, ref, tol, "y")


@pytest.mark.parametrize("D,page,dtype", [(128, 16, torch.bfloat16), (256, 7, torch.bfloat16), (64, 16, torch.float32)])
@pytest.mark.parametrize("window", [0, 33])
def test_the_rows_of_a_chunk_as_sequences_that_share_pages(D, page, dtype, window):
    """Row i behind a prefix: a sequence of its own with nonpad = its position + 1."""
    n, first = 100, 61
    _, k, v, table, _ = paged.make((n,), 8, 2, D, page, dtype)
    lens = tuple(range(first, n + 1))
    gen = torch.Generator().manual_seed(4)
    q = torch.randn((len(lens), 8, D), generator=gen).to(dtype).cuda()
    tables = table.expand(len(lens), -1).contiguous()
    y = paged.run(q, k, v, tables, torch.tensor(lens, device="cuda"), 0.1, window)
    ref, tol = paged.reference(q, k, v, tables, lens, window, 0.1)
    packed_ref.check(y, ref, tol, "chunk")
