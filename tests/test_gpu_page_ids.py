"""Page ids below zero, whatever their value, are flagged and their keys left out: by every
kernel that looks a page up, on the tables of the sequences and of the prefixes."""
import pytest
import torch

import test_gpu_fp8_pages as fp8
import test_gpu_paged_decode as pages
import test_gpu_shared_prefix as shared
from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WRONG = (-2, -3, -(1 << 62))
LENS = (100, 40, 64, 200)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def flagged(st, what):
    assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE and int(st[0]) == ek.EXTKV_DEV_BAD_PAGE, (what, int(st[0]))


@pytest.mark.parametrize("algo", [ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO], ids=["axis", "auto"])
@pytest.mark.parametrize("D,page,dtype", [(64, 32, BF), (128, 16, BF), (256, 16, BF), (512, 48, BF), (128, 7, BF), (64, 16, F32)],
                         ids=lambda x: str(x))
def test_paged_decode(D, page, dtype, algo):
    q, k, v, table, nonpad = pages.make(LENS, 4, 2, D, page, dtype)
    last = (LENS[3] - 1) // page  # the last sequence's last page, so that what is left is a shorter sequence
    ref, tol = pages.reference(q, k, v, table, (*LENS[:3], last * page), 0, 0.1)
    for wrong in WRONG:
        table[3, last] = wrong
        y, st = torch.full_like(q, 7.0), ek.new_status()
        with ek.use_algo(algo):
            ek.attention_paged_decode(y, q, k, v, table, nonpad, 0.1, status=st)
        check(y, ref, tol, f"page {wrong}")
        flagged(st, wrong)


@pytest.mark.parametrize("algo", [ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO], ids=["axis", "auto"])
@pytest.mark.parametrize("D,page,dtype", [(256, 32, BF), (512, 16, BF), (256, 64, F32), (128, 16, BF), (96, 16, BF)],
                         ids=lambda x: str(x))
def test_decode_over_codes(D, page, dtype, algo):
    q, k, v, sc, table, nonpad = fp8.make(LENS, 4, 2, D, page, dtype)
    ref, tol = fp8.reference(q, k, v, sc, table, LENS, 0, 0.1, lambda b, j: (j // page != 1) | (b != 3))
    for wrong in WRONG:
        table[3, 1] = wrong
        y, st = torch.full_like(q, 7.0), ek.new_status()
        with ek.use_algo(algo):
            ek.attention_paged_decode_fp8(y, q, k, v, sc, table, nonpad, 0.1, status=st)
        check(y, ref, tol, f"page {wrong}")
        flagged(st, wrong)


@pytest.mark.parametrize("wide", [0, 4000], ids=["", "wide_front"])  # (D = 128: own pages beside the prefix, and after it)
@pytest.mark.parametrize("D,page,dtype", [(64, 64, BF), (128, 16, BF), (128, 32, BF), (256, 32, BF), (128, 7, BF), (64, 16, F32)],
                         ids=lambda x: str(x))
def test_shared_prefix(D, page, dtype, wide):
    s = shared.make((200, 130), (60, 2), (30, 1, 0, 64) * 15 + (64, 9), 8, 2, D, page, dtype)
    old = s["front"]
    s["front"] = torch.full((2, old.shape[1] + wide), -1, dtype=torch.int64, device="cuda")
    s["front"][:, :old.shape[1]] = old
    front = shared.reference(s, 0.1, keep=lambda kind, b, j: (j // page != 2) | (kind != "prefix") | (b != 0))
    own = shared.reference(s, 0.1, keep=lambda kind, b, j: (j // page != 0) | (kind != "own") | (b != 3))
    for wrong in WRONG:
        for name, at, (ref, tol) in (("front", (0, 2), front), ("table", (3, 0), own)):
            good = int(s[name][at])
            s[name][at] = wrong
            st = ek.new_status()
            y = shared.run(s, 0.1, status=st)
            check(y, ref, tol, f"{name}: page {wrong}")
            flagged(st, (name, wrong))
            s[name][at] = good


def test_rows_in_and_out():
    """The append and the way back leave out the rows of such a page, and flag it."""
    k, v, sc = ek.new_fp8_pages(3, 2, 16, 64)
    kp, vp = (torch.zeros((3, 2, 16, 64), dtype=BF, device="cuda") for _ in range(2))
    rows = torch.randn((20, 2, 64), device="cuda").to(BF)
    zero, cu = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor([0, 20], device="cuda")
    for wrong in WRONG:
        table = torch.tensor([[1, wrong]], device="cuda")
        st = ek.new_status()
        ek.paged_kv_append(kp, vp, rows, rows, table, zero, cu_seqlens=cu, status=st)
        flagged(st, wrong)
        assert torch.equal(kp[1].transpose(0, 1), rows[:16])
        st = ek.new_status()
        ek.paged_kv_append_fp8(k, v, sc, rows, rows, table, zero, cu_seqlens=cu, status=st)
        flagged(st, wrong)
        out, st = torch.full_like(rows, 7.0), ek.new_status()
        ek.paged_kv_read_fp8(out, out.clone(), k, v, sc, table, zero, cu_seqlens=cu, status=st)
        flagged(st, wrong)
        assert bool((out[16:] == 7).all()) and not bool((out[:16] == 7).all())
