"""The packed and paged attention kernels when a pipeline wait gives up: every
poll limit, from none to one that some waits meet and others do not, leaves a
context in which the next call has the right bits.  A wait that gives up
leaves copies in flight, and the warps of a CTA learn of it at different times;
all lanes of a warp leave its loop together, and the copies land before the
CTA leaves.  Nothing here faults, traps or hangs the GPU: each wait is bounded
and the kernels end by themselves."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
import test_gpu_packed_prefill as packed
import test_gpu_paged_decode as paged

pytestmark = pytest.mark.gpu

LIMITS = (0, 1, 2, 7, 40, 65, 150, 400, 2000)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def give_up(call, status, y, good, what):
    """`call` under every limit, several times; in between a call whose waits are met."""
    gave_up = 0
    for limit in LIMITS:
        for _ in range(6):
            status.zero_()
            with ek.wait_polls(limit):
                call()
            code = ek.extkv_read_status(status)
            if code != ek.EXTKV_OK:
                assert int(status[0]) == ek.EXTKV_DEV_TIMEOUT, (what, limit, int(status[0]))
                gave_up += 1
            else:
                assert torch.equal(y, good), (what, limit)  # no wait gave up: whole
            status.zero_()
            y.fill_(7.0)
            call()
            assert ek.extkv_read_status(status) == ek.EXTKV_OK, ek.extkv_last_error()
            assert torch.equal(y, good), (what, limit)
    assert gave_up >= 6, what  # with no poll at all every call gives up


@pytest.mark.parametrize("algo", [ek.ALGO_DECODE_STREAMK, ek.ALGO_DECODE_CLUSTER], ids=["axis", "cluster"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ((17,), 4, 2, 64, 16),                  # fewer tiles than ring slots: the producer is done before a consumer starts
    ((300, 77, 0, 5000), 4, 2, 128, 16),
    ((900, 33), 16, 1, 256, 48),
    ((1000, 1, 260), 8, 2, 512, 32),
], ids=lambda x: str(x))
def test_paged_decode_gives_up_cleanly(lens, Hq, Hkv, D, page, algo):
    scale = 1.0 / math.sqrt(D)
    q, k, v, table, nonpad = paged.make(lens, Hq, Hkv, D, page, torch.bfloat16)
    with ek.use_algo(algo):
        good = paged.run(q, k, v, table, nonpad, scale, 0)
        y, st = torch.empty_like(good), ek.new_status()
        give_up(lambda: ek.attention_paged_decode(y, q, k, v, table, nonpad, scale, status=st), st, y, good,
                (lens, D, algo))


@pytest.mark.parametrize("lens,Hq,Hkv,D,window", [
    ((20,), 4, 2, 64, 0),
    ((1, 0, 129, 700), 8, 4, 128, 0),
    ((2047,), 8, 4, 128, 0),                # items whose keys are split over the CTA's two query tiles
    ((900, 33, 128), 4, 2, 64, 100),
    ((5,), 2, 1, 256, 0),
    ((700, 1, 300), 4, 2, 256, 200),
], ids=lambda x: str(x))
def test_packed_prefill_gives_up_cleanly(lens, Hq, Hkv, D, window):
    scale = 1.0 / math.sqrt(D)
    q, k, v, cu = packed.make(lens, Hq, Hkv, D, torch.bfloat16)
    good = packed.run(q, k, v, cu, scale, True, window)
    assert ek.extkv_last_kernel() == "packed_tcgen05"
    y, st = torch.empty_like(good), ek.new_status()
    give_up(lambda: ek.attention_packed_prefill(y, q, k, v, cu, scale, window=window, status=st), st, y, good, (lens, D))
