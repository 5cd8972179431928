"""attention_shared_prefix_decode where own slots could be attended beside the prefix and are
attended after it (a wide prefix table): which calls do, against the definition, between guard regions, on one
workspace in turn with calls that attend them beside, with a wait that gives up, and on the
library with bounds checks."""
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
from test_gpu_paged_timeout import give_up
from test_gpu_shared_prefix import args, make, reference, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HERE = os.path.dirname(os.path.abspath(__file__))
BESIDE, AFTER = "shared_prefix_tcgen05", "shared_prefix_tcgen05_after"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def wide(s, pages=16000):
    """The same keys by a prefix table of `pages` more pages."""
    old = s["front"]
    s["front"] = torch.full((old.shape[0], old.shape[1] + pages), -1, dtype=torch.int64, device="cuda")
    s["front"][:, :old.shape[1]] = old
    return s


def lens(B):
    return tuple((31 * i) % 97 for i in range(B))


@pytest.mark.parametrize("Hq,Hkv,D,B,after", [(8, 2, 128, 40, AFTER), (12, 4, 128, 70, AFTER), (8, 1, 128, 33, AFTER),
                                              (8, 2, 128, 6, BESIDE),    # few rows: beside
                                              (64, 2, 128, 40, BESIDE),  # more than 8 heads a KV head, or another head size: always after
                                              (8, 2, 64, 40, BESIDE), (8, 2, 256, 40, BESIDE)], ids=lambda x: str(x))
def test_which_calls(Hq, Hkv, D, B, after):
    s = make((700,), (B,), lens(B), Hq, Hkv, D, 16, BF)
    ref, tol = reference(s, 0.08)
    check(run(s, 0.08), ref, tol, "narrow")
    assert ek.extkv_last_kernel() == BESIDE
    check(run(wide(s), 0.08), ref, tol, "wide")
    assert ek.extkv_last_kernel() == after


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("page", [16, 64])
def test_between_guards(page, window):
    s = wide(make((700, 33), (90, 1), lens(92), 8, 2, 128, page, BF, window=window))
    y = Guarded(tuple(s["q"].shape), BF)
    n = ek.attention_shared_prefix_decode_workspace_size(92, 2, 8, 2, 128, BF)
    ws, st = Guarded((n,), torch.uint8), guarded_status()
    ek.attention_shared_prefix_decode(y.view, *(between(t) for t in args(s)), 0.1, window=window, workspace=ws.view, status=st.view)
    assert ek.extkv_read_status(st.view) == ek.EXTKV_OK, ek.extkv_last_error()
    assert ek.extkv_last_kernel() == AFTER
    intact(y=y, workspace=ws, status=st)
    ref, tol = reference(s, 0.1, window)
    check(y.view, ref, tol, "y")


def test_gives_up_cleanly():
    s = wide(make((700,), (60,), (5,) * 60, 8, 2, 128, 16, BF))
    good = run(s, 0.1)
    assert ek.extkv_last_kernel() == AFTER
    y, st = torch.empty_like(good), ek.new_status()
    give_up(lambda: ek.attention_shared_prefix_decode(y, *args(s), 0.1, status=st), st, y, good, "after")


def test_in_turn_on_one_workspace():
    """Both ways lay the workspace out differently: neither leaves what the other would read."""
    a = make((700,), (40,), lens(40), 8, 2, 128, 16, BF)
    b = wide(make((900, 70), (60, 5), lens(65), 16, 4, 128, 64, BF, seed=1))
    need = max(ek.attention_shared_prefix_decode_workspace_size(*n, BF) for n in ((40, 1, 8, 2, 128), (65, 2, 16, 4, 128)))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    good = []
    for s, name in ((a, BESIDE), (b, AFTER)):
        good.append(run(s, 0.08))
        assert ek.extkv_last_kernel() == name
        ref, tol = reference(s, 0.08)
        check(good[-1], ref, tol, name)
    out = [torch.zeros_like(g) for g in good]
    st, stream = ek.new_status(), torch.cuda.Stream()

    def both():
        for y, s in zip(out, (a, b)):
            ek.attention_shared_prefix_decode(y, *args(s), 0.08, workspace=ws, status=st, stream=torch.cuda.current_stream())

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(20):
            both()
    stream.synchronize()
    for y, g in zip(out, good):
        assert torch.equal(y, g)
        y.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        both()
        both()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for y, g in zip(out, good):
        assert torch.equal(y, g)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK


def test_with_bounds_checks():
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_after_run.py")], capture_output=True, text=True,
                       timeout=1800, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, (r.stdout[-3000:] + r.stderr[-3000:])
    assert "checked ok" in r.stdout, r.stdout[-2000:]
