"""Pages of more slots than 2^24, so that a slot's offset in its page, in bytes, passes 2^31:
windows at their ends, over pages that requests load and over rows that warps copy."""
import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from fp8_ref import decode_rows, values
from packed_ref import attention_rows, bound, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
WINDOW = 300


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("extra", [32, 33], ids=["requests", "copies"])
def test_paged_and_shared_prefix(extra):
    D, page = 64, (1 << 24) + extra
    n = page - 5
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.full((1, 1, page, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    for t in (k, v):
        t[0, 0, n - WINDOW:n] = torch.randn((WINDOW, D), generator=gen, device="cuda").to(BF)
    q = torch.randn((1, 4, D), generator=gen, device="cuda").to(BF)
    table, nonpad = torch.zeros((1, 1), dtype=torch.int64, device="cuda"), torch.tensor([n], device="cuda")
    ok = torch.ones((4, WINDOW), dtype=torch.bool, device="cuda")
    ref, pv, size = attention_rows(q[0], k[0, 0, n - WINDOW:n], v[0, 0, n - WINDOW:n], ok, 0.1)
    tol = bound(ref, pv, size, D, WINDOW, BF, True)
    for algo in (ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO):
        y, st = torch.empty_like(q), ek.new_status()
        with ek.use_algo(algo):
            ek.attention_paged_decode(y, q, k, v, table, nonpad, 0.1, window=WINDOW, status=st)
        assert ek.extkv_read_status(st) == ek.EXTKV_OK
        check(y[0], ref, tol, "paged")
    # the same keys as a prefix, and as the slots behind an empty one
    zero, cu = torch.zeros_like(nonpad), torch.tensor([0, 1], device="cuda")
    for plen, own in ((nonpad, zero), (zero, nonpad)):
        y, st = torch.empty_like(q), ek.new_status()
        ek.attention_shared_prefix_decode(y, q, k, v, table, plen, cu, table, own, 0.1, window=WINDOW, status=st)
        assert ek.extkv_read_status(st) == ek.EXTKV_OK
        check(y[0], ref, tol, "shared prefix")


@pytest.mark.parametrize("extra", [32, 33], ids=["requests", "copies"])
def test_codes(extra):
    D, page = 256, (1 << 24) + extra
    n = page - 5
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.full((1, 1, page, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.full((1, 1, page, 2), 255, dtype=torch.uint8, device="cuda")
    k8, v8 = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    table, nonpad = torch.zeros((1, 1), dtype=torch.int64, device="cuda"), torch.tensor([n], device="cuda")
    new = [torch.randn((WINDOW, 1, D), generator=gen, device="cuda").to(BF) for _ in range(2)]
    cu, st = torch.tensor([0, WINDOW], device="cuda"), ek.new_status()
    ek.paged_kv_append_fp8(k8, v8, sc, *new, table, nonpad - WINDOW, cu_seqlens=cu, status=st)
    at = slice(n - WINDOW, n)
    kd, vd = (values(t[0, 0, at], sc[0, 0, at, i]) for i, t in enumerate((k, v)))
    back = [torch.empty_like(x) for x in new]
    ek.paged_kv_read_fp8(*back, k8, v8, sc, table, nonpad - WINDOW, cu_seqlens=cu, status=st)
    assert torch.equal(back[0][:, 0].double(), kd) and torch.equal(back[1][:, 0].double(), vd)
    q = torch.randn((1, 4, D), generator=gen, device="cuda").to(BF)
    ok = torch.ones((4, WINDOW), dtype=torch.bool, device="cuda")
    ref, tol = decode_rows(q[0], kd, vd, sc[0, 0, at, 1].double() - 127, ok, 0.1, BF, True)
    for algo in (ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO):
        y = torch.empty_like(q)
        with ek.use_algo(algo):
            ek.attention_paged_decode_fp8(y, q, k8, v8, sc, table, nonpad, 0.1, window=WINDOW, status=st)
        check(y[0], ref, tol, "codes")
    assert ek.extkv_read_status(st) == ek.EXTKV_OK
