"""attention_shared_prefix_decode with windows that begin inside the prefix: an infinity or a NaN
in a row of V or K reaches the sequences that attend that slot, and none of the others of their
group, whose results are those of finite pages."""
import math
import os
import subprocess
import sys

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check
from test_gpu_canaries import Guarded
from test_gpu_fp8_canaries import between
from test_gpu_paged_canaries import guarded_status, intact
from test_gpu_shared_prefix import args, live_from, make, reference, run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def poison(s, spots):
    """Writes `spots` ((K or V, prefix, slot, KV head, column, value)); returns the references that they leave and,
    for each, the rows and columns that attend it."""
    g, page = s["q"].shape[1] // s["k"].shape[1], s["k"].shape[2]
    for name, o, j, h, c, value in spots:
        s[name][int(s["front"][o, j // page]), h, j % page, c] = value
    return [(name, o, j, slice(h * g, h * g + g), c) for name, o, j, h, c, _ in spots]


def expect(s, y, ref, tol, hit, window):
    where = torch.zeros(y.shape, dtype=torch.bool, device="cuda")
    for name, o, j, heads, c in hit:
        for b, n in enumerate(s["lens"]):
            if s["owner"][b] == o and live_from(s["plens"][o], n, window)[0] <= j:
                where[b, heads, c if name == "v" else slice(None)] = True
    assert bool(where.any()) and not bool(torch.isfinite(y[where].float()).any())
    check(torch.where(where, ref, y.double()), ref, tol, "the rest")
    return where


# own lengths from none to more than the window: sequences that attend all of it, a part, nothing
MIXED = (1, 60, 9, 200, 0, 149, 150, 33)
CASES = [  # prefix, group sizes, own lengths, Hq, Hkv, D, page, window, dtype
    ((200, 64), (7, 1), MIXED, 4, 2, 128, 16, 150, BF),
    ((200, 64), (7, 1), MIXED, 8, 2, 64, 64, 150, BF),
    ((200, 64), (7, 1), MIXED, 6, 2, 256, 16, 150, BF),
    ((200, 64), (7, 1), MIXED, 16, 2, 512, 16, 150, BF),
    ((200, 64), (7, 1), MIXED, 4, 2, 128, 7, 150, BF),
    ((200, 64), (7, 1), MIXED, 4, 2, 96, 16, 150, BF),
    ((200, 64), (7, 1), MIXED, 4, 2, 64, 16, 150, F32),
    ((200, 64), (7, 1), MIXED, 2, 1, 512, 16, 150, F32),
    ((3000, 64), (130, 1), tuple((37 * i) % 900 for i in range(131)), 8, 2, 128, 16, 1000, BF),   # a warp a row in the join
    ((3000, 64), (130, 1), tuple((37 * i) % 900 for i in range(131)), 8, 2, 64, 16, 1000, BF),
    ((3000, 64), (90, 1), tuple((37 * i) % 900 for i in range(91)), 8, 2, 256, 32, 1000, BF),
    ((900, 64), (130, 1), tuple((37 * i) % 400 for i in range(131)), 8, 2, 512, 16, 500, BF),
    ((900, 64), (130, 1), tuple((37 * i) % 400 for i in range(131)), 8, 2, 48, 16, 500, F32),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"P{max(c[0])}B{len(c[2])}_h{c[3]}-{c[4]}_d{c[5]}_p{c[6]}_w{c[7]}_{str(c[8])[6:]}")
def test_sequences_that_do_not_attend_it_are_whole(case):
    prefix, sizes, lens, Hq, Hkv, D, page, window, dtype = case
    s = make(prefix, sizes, lens, Hq, Hkv, D, page, dtype, window=window)
    scale, P = 1.0 / math.sqrt(D), prefix[0]
    ref, tol = reference(s, scale, window)  # (of those that do not attend a spot)
    h = Hkv - 1
    spots = [("v", 0, P - window + 70, h, 5, math.inf), ("v", 0, P - window + 71, h, D - 1, -math.inf), ("v", 0, P - 3, 0, 0, math.nan)]
    hit = poison(s, spots)
    y = run(s, scale, window)
    where = expect(s, y, ref, tol, hit, window)
    rows = where.any(2).any(1)
    assert not bool(rows.all()) and bool(rows.any())
    assert bool((y[..., 5][where[..., 5] & ~where[..., 4]] == math.inf).all())
    assert torch.equal(y.view(torch.uint8), run(s, scale, window).view(torch.uint8))
    hit += poison(s, [("k", 0, P - window + 65, h, 3, math.nan)])
    expect(s, run(s, scale, window), ref, tol, hit, window)


def test_with_a_bad_page_besides():
    s = make((200,), (7,), MIXED[:7], 4, 2, 128, 16, BF, window=150)
    keep = lambda kind, b, j: (j // 16 != 8) | (kind != "prefix")  # noqa: E731
    ref, tol = reference(s, 0.1, 150, keep)
    hit = poison(s, [("v", 0, 100, 1, 5, math.inf)])
    s["front"][0, 8] = -1
    st = ek.new_status()
    y = run(s, 0.1, 150, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE and int(st[0]) == ek.EXTKV_DEV_BAD_PAGE
    expect(s, y, ref, tol, hit, 150)


@pytest.mark.parametrize("D,dtype,q_gap", [(128, BF, 0), (128, BF, 72), (96, BF, 8), (64, F32, 4)])
def test_between_guards_and_recorded(D, dtype, q_gap):
    s = make((200, 64), (7, 1), MIXED, 8, 2, D, 16, dtype, window=150, q_gap=q_gap)
    ref, tol = reference(s, 0.1, 150)
    hit = poison(s, [("v", 0, 120, 1, 5, math.nan)])
    y = Guarded(tuple(s["q"].shape), dtype)
    ws = Guarded((ek.attention_shared_prefix_decode_workspace_size(8, 2, 8, 2, D, dtype),), torch.uint8)
    st = guarded_status()
    rest = args(s)[1:]
    q = s["q"] if q_gap else between(s["q"])
    ek.attention_shared_prefix_decode(y.view, q, *(between(t) for t in rest), 0.1, window=150, workspace=ws.view, status=st.view)
    assert ek.extkv_read_status(st.view) == ek.EXTKV_OK, ek.extkv_last_error()
    intact(y=y, workspace=ws, status=st)
    expect(s, y.view, ref, tol, hit, 150)
    z = torch.zeros_like(y.view)
    with ek.StepRecorder() as rec:
        ek.attention_shared_prefix_decode(z, *args(s), 0.1, window=150, stream=rec.stream)
    rec.step(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(z.view(torch.uint8), y.view.view(torch.uint8))


def test_with_bounds_checks():
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_isolation_run.py")], capture_output=True, text=True,
                       timeout=1800, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "checked ok" in r.stdout, r.stdout[-2000:]
