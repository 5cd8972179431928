"""Infinities and NaN in live slots: they reach the rows that attend them, in the columns where
the definition has them, and no other head or column, nor any other sequence's rows (those of a
prefix' group whose window leaves the slot out: test_gpu_window_isolation.py)."""
import math

import pytest
import torch

import test_gpu_fp8_pages as fp8
import test_gpu_paged_decode as pages
import test_gpu_shared_prefix as shared
from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan
NAN_CODE = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


@pytest.fixture(params=[ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO], ids=["axis", "auto"])
def each_kernel(request):
    with ek.use_algo(request.param):
        yield


def same_kind(got, want):
    """Infinities of one sign, or NaN."""
    return bool(torch.isnan(got).all()) if math.isnan(want) else bool((got == want).all())


def rest(y, ref, tol, where, what):
    """All of y but `where` (a mask) within its bound."""
    check(torch.where(where, ref, y.double()), ref, tol, what)


LENS = (300, 0, 77)


@pytest.mark.parametrize("D,page,dtype", [(64, 16, BF), (128, 16, BF), (256, 32, BF), (256, 7, BF), (512, 16, BF), (96, 16, BF),
                                          (128, 16, F32), (256, 32, F32), (48, 16, F32)], ids=lambda x: str(x))
def test_codes(D, page, dtype, each_kernel):
    q, k, v, sc, table, nonpad = fp8.make(LENS, 4, 2, D, page, dtype)
    at = int(table[0, 123 // page]), 1, 123 % page  # a slot of the first sequence, KV head 1: query heads 2 and 3
    for pool, column in ((v, 5), (v, D - 1), (k, 9)):
        raw = pool.view(torch.uint8)
        old = int(raw[(*at, column)])
        raw[(*at, column)] = 0
        ref, tol = fp8.reference(q, k, v, sc, table, LENS, 0, 0.1)
        raw[(*at, column)] = NAN_CODE
        y = fp8.run(q, k, v, sc, table, nonpad, 0.1, 0)
        where = torch.zeros_like(y, dtype=torch.bool)
        where[0, 2:4, column if pool is v else slice(None)] = True  # (of K: every weight of the row)
        assert bool(torch.isnan(y[where]).all())
        rest(y, ref, tol, where, "codes")
        raw[(*at, column)] = old


@pytest.mark.parametrize("D,page,dtype", [(64, 16, BF), (128, 7, BF), (512, 16, BF), (96, 16, BF), (128, 16, F32)], ids=lambda x: str(x))
def test_pages(D, page, dtype, each_kernel):
    q, k, v, table, nonpad = pages.make(LENS, 4, 2, D, page, dtype)
    at = int(table[0, 123 // page]), 1, 123 % page
    for pool, column, value in ((v, 5, INF), (v, D - 1, -INF), (v, 0, NAN), (k, 7, NAN)):
        old = float(pool[(*at, column)])
        pool[(*at, column)] = 0.0
        ref, tol = pages.reference(q, k, v, table, LENS, 0, 0.1)
        pool[(*at, column)] = value
        y = pages.run(q, k, v, table, nonpad, 0.1, 0)
        where = torch.zeros_like(y, dtype=torch.bool)
        where[0, 2:4, column if pool is v else slice(None)] = True
        assert same_kind(y[where], value)
        rest(y, ref, tol, where, "pages")
        pool[(*at, column)] = old


SHARED = [(64, 16, BF), (128, 16, BF), (128, 64, BF), (256, 32, BF), (512, 16, BF), (128, 7, BF), (96, 16, BF), (64, 16, F32)]


@pytest.mark.parametrize("D,page,dtype", SHARED, ids=lambda x: str(x))
@pytest.mark.parametrize("window", [0, 150])
def test_shared_prefix(D, page, dtype, window):
    """With the window the sequences begin at slots 51, 110, 59 of the first prefix."""
    lens = (1, 60, 9, 40)
    s = shared.make((200, 64), (3, 1), lens, 4, 2, D, page, dtype, window=window)
    attends = torch.tensor([True, window == 0, True, False], device="cuda")
    at = int(s["front"][0, 70 // page]), 1, 70 % page
    for name, column, value in (("v", 5, INF), ("v", D - 1, -INF), ("v", 0, NAN), ("k", 7, NAN)):
        pool = s[name]
        old = float(pool[(*at, column)])
        pool[(*at, column)] = 0.0
        ref, tol = shared.reference(s, 0.1, window)
        pool[(*at, column)] = value
        y = shared.run(s, 0.1, window)
        cols = column if name == "v" else slice(None)
        where = torch.zeros_like(y, dtype=torch.bool)
        where[attends, 2:4, cols] = True
        assert same_kind(y[where], value)
        if name == "v":
            where[:3, 2:4, cols] = True
        rest(y, ref, tol, where, f"prefix {name}")
        pool[(*at, column)] = old
    # in a sequence's own slots: its rows alone
    at = int(s["table"][1, 33 // page]), 0, 33 % page
    for name, column, value in (("v", 5, INF), ("k", 7, NAN)):
        pool = s[name]
        old = float(pool[(*at, column)])
        pool[(*at, column)] = 0.0
        ref, tol = shared.reference(s, 0.1, window)
        pool[(*at, column)] = value
        y = shared.run(s, 0.1, window)
        where = torch.zeros_like(y, dtype=torch.bool)
        where[1, 0:2, column if name == "v" else slice(None)] = True
        assert same_kind(y[where], value)
        rest(y, ref, tol, where, f"own {name}")
        pool[(*at, column)] = old


@pytest.mark.parametrize("D,page,dtype", SHARED, ids=lambda x: str(x))
def test_a_window_that_no_row_begins_inside(D, page, dtype):
    """Slots in front of every row's window are nobody's, whatever their tile holds besides."""
    lens = (9, 9, 9)
    s = shared.make((200,), (3,), lens, 4, 2, D, page, dtype, window=150)  # from slot 59 on
    ref, tol = shared.reference(s, 0.1, 150)
    for j in (0, 58):
        at = int(s["front"][0, j // page]), slice(None), j % page
        assert bool(torch.isnan(s["v"][at]).all())  # (as make leaves them)
        for value in (INF, -INF):
            s["k"][at], s["v"][at] = value, value
            check(shared.run(s, 0.1, 150), ref, tol, f"slot {j}")
