"""attention_shared_prefix_decode with more groups than a warp has lanes, whose sums lie in shared
memory where the first row tile's queries come next: the same bits call after call, with
other work between the calls and without, and the definition's values."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check
from test_gpu_shared_prefix import args, make, reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("G,g,Hkv,D", [(32, 4, 1, 128), (33, 8, 2, 64), (64, 1, 2, 256), (129, 2, 1, 128), (500, 1, 1, 64), (40, 3, 1, 128)])
def test_more_groups_than_lanes(G, g, Hkv, D):
    sizes = tuple(1 + (5 * i) % 3 for i in range(G))
    prefix = tuple((37 * i) % 150 for i in range(G))
    s = make(prefix, sizes, tuple((7 * i) % 20 for i in range(sum(sizes))), g * Hkv, Hkv, D, 16, BF)
    scale = 1.0 / math.sqrt(D)
    y = torch.empty_like(s["q"])
    call = ek.prepare_attention_shared_prefix_decode(y, *args(s), scale)
    call()
    ref, tol = reference(s, scale)
    check(y, ref, tol, "y")
    good, other = y.clone(), torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for i in range(40):
        y.fill_(7.0)
        if i & 1:
            other.fill_(i)
        for _ in range(1 + i % 3):
            call()
        assert torch.equal(y, good), i
