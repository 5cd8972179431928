"""The axis of tiles cut over CTAs and warps, at the counts where the cut changes:
one tile a CTA, one tile a warp, one more and one less, and several a warp.
Warps a CTA and keys a tile are the kernel's, by head size."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check
import test_gpu_paged_decode as paged

pytestmark = pytest.mark.gpu

# head size: (warps that take tiles, keys of a tile) of the tensor-core kernels
SHAPES = {64: (6, 32), 128: (6, 32), 256: (4, 16), 512: (6, 16)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def tile_counts(sms, warps):
    w = sms * warps
    return sorted({1, 2, sms - 1, sms, sms + 1, 2 * sms, w - 1, w, w + 1, 2 * w, 5 * w + 3})


@pytest.mark.parametrize("page", [64, 7], ids=["tma", "copies"])
@pytest.mark.parametrize("D", sorted(SHAPES))
@pytest.mark.parametrize("nth", range(11))
def test_one_sequence_of_so_many_tiles(D, page, nth):
    warps, keys = SHAPES[D]
    tiles = tile_counts(torch.cuda.get_device_properties(0).multi_processor_count, warps)[nth]
    scale = 1.0 / math.sqrt(D)
    for n in {tiles * keys, (tiles - 1) * keys + 1}:  # a last tile that is full, and one of a single key
        q, k, v, table, nonpad = paged.make((n,), 4, 1, D, page, torch.bfloat16)
        with ek.use_algo(ek.ALGO_DECODE_STREAMK):
            y = paged.run(q, k, v, table, nonpad, scale, 0)
        assert ek.extkv_last_kernel() == "paged_decode_mma"
        ref, tol = paged.reference(q, k, v, table, (n,), 0, scale)
        check(y, ref, tol, f"{n} keys")
        # the bound above grows with the number of keys; independent roundings do not
        # (P's and the result's, 2^-8 of each weight and of each element at most)
        assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -7


@pytest.mark.parametrize("D", sorted(SHAPES))
@pytest.mark.parametrize("extra", [-1, 0, 1])
def test_units_of_one_tile_each(D, extra):
    """As many units as CTAs or warps: every unit begins and ends in one part, or next to one."""
    warps, keys = SHAPES[D]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for units in (sms + extra, sms * warps + extra):
        lens = tuple(1 + (7 * i) % keys for i in range(units))
        scale = 1.0 / math.sqrt(D)
        q, k, v, table, nonpad = paged.make(lens, 2, 1, D, 32, torch.bfloat16)
        with ek.use_algo(ek.ALGO_DECODE_STREAMK):
            y = paged.run(q, k, v, table, nonpad, scale, 0)
        ref, tol = paged.reference(q, k, v, table, lens, 0, scale)
        check(y, ref, tol, f"{units} units")


def test_the_shapes_are_the_kernels():
    """SHAPES as the launch in the source names them: <D, head groups, keys, slots, warps>."""
    import os
    import re
    from biased_gqa_attention_gb300 import build
    src = open(os.path.join(build.CSRC, "paged_decode.cu")).read()
    named = {(int(d), int(w), int(kt)) for d, kt, w in re.findall(r"launch_mma<(\d+), [12], (\d+), \d+, (\d+)>\(p", src)}
    assert named == {(d, w, kt) for d, (w, kt) in SHAPES.items()}
