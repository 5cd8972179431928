"""attention_packed_prefill against the definition in 64 bits: empty and
one-token sequences, lengths around the tile sizes, rows outside every
sequence, slices of one projection, causal and not, windows, every head group."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import attention_rows, bound, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def make(lens, Hq, Hkv, D, dtype, fused=False, before=0, behind=0, seed=0, sigma=2.0):
    """Inputs with `before` and `behind` rows outside every sequence, NaN there."""
    gen = torch.Generator().manual_seed(77 + seed)
    T = before + sum(lens) + behind
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen, dtype=torch.float32)
    x[:, :Hq] *= sigma
    x[:before] = float("nan")
    if behind:
        x[-behind:] = float("nan")
    x = x.to(dtype).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        q, k, v = (t.contiguous() for t in (q, k, v))
    cu = [before]
    for n in lens:
        cu.append(cu[-1] + n)
    return q, k, v, torch.tensor(cu, dtype=torch.int64).cuda()


def fast(D, dtype):
    return dtype == torch.bfloat16 and D in (64, 128, 256)


def reference(q, k, v, cu, scale, causal, window):
    T, Hq, D = q.shape
    g = Hq // k.shape[1]
    y = torch.full((T, Hq, D), 7.0, dtype=torch.float64, device=q.device)
    tol = torch.full_like(y, 1e-30)
    cu = cu.tolist()
    for a, b in zip(cu, cu[1:]):
        n = b - a
        i = torch.arange(n, device=q.device)
        ok = torch.ones((n, n), dtype=torch.bool, device=q.device)
        if causal:
            ok &= i[None, :] <= i[:, None]
        if window > 0:
            ok &= i[:, None] - i[None, :] < window
        for h in range(Hq):
            o, pv, size = attention_rows(q[a:b, h], k[a:b, h // g], v[a:b, h // g], ok, scale)
            y[a:b, h] = o
            tol[a:b, h] = bound(o, pv, size, D, n, q.dtype, fast(D, q.dtype))
    return y, tol


def run(q, k, v, cu, scale, causal, window, **kw):
    y = torch.full(q.shape, 7.0, dtype=q.dtype, device=q.device)
    st = ek.new_status()
    ek.attention_packed_prefill(y, q, k, v, cu, scale, causal=causal, window=window, status=st, **kw)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK, ek.extkv_last_error()
    return y


EDGES = (1, 0, 127, 128, 129, 2, 0, 255, 257, 64, 300)
CASES = [
    # lens, Hq, Hkv, D, dtype, causal, window, fused, before, behind
    (EDGES, 8, 4, 128, torch.bfloat16, True, 0, False, 0, 0),
    (EDGES, 8, 4, 128, torch.bfloat16, True, 0, True, 3, 5),
    (EDGES, 8, 4, 128, torch.bfloat16, False, 0, False, 1, 200),
    (EDGES, 8, 4, 128, torch.bfloat16, True, 100, True, 0, 0),
    (EDGES, 8, 4, 128, torch.bfloat16, True, 1, False, 0, 1),
    (EDGES, 4, 2, 128, torch.bfloat16, False, 130, False, 0, 0),
    (EDGES, 4, 4, 128, torch.bfloat16, True, 0, False, 0, 0),
    (EDGES, 6, 2, 128, torch.bfloat16, True, 0, True, 0, 0),
    (EDGES, 12, 2, 128, torch.bfloat16, True, 70, False, 0, 0),
    (EDGES, 16, 1, 128, torch.bfloat16, True, 0, False, 0, 0),
    (EDGES, 5, 1, 64, torch.bfloat16, True, 0, False, 2, 2),
    (EDGES, 8, 1, 64, torch.bfloat16, False, 0, True, 0, 0),
    (EDGES, 16, 8, 256, torch.bfloat16, True, 0, False, 0, 0),
    (EDGES, 16, 8, 256, torch.bfloat16, True, 90, True, 4, 4),
    (EDGES, 3, 1, 256, torch.bfloat16, False, 0, False, 0, 0),
    (EDGES, 8, 1, 256, torch.bfloat16, True, 0, False, 0, 0),
    (EDGES, 4, 2, 96, torch.bfloat16, True, 0, True, 3, 3),
    (EDGES, 4, 2, 512, torch.bfloat16, True, 50, False, 0, 0),
    (EDGES, 4, 2, 64, torch.float32, True, 0, False, 0, 0),
    (EDGES, 6, 2, 128, torch.float32, False, 0, True, 3, 3),
    (EDGES, 4, 1, 264, torch.float32, True, 40, False, 0, 0),
    ((5, 0, 33, 2), 128, 1, 64, torch.bfloat16, True, 0, True, 0, 3),     # a token a query tile
    ((5, 0, 33, 2), 64, 2, 256, torch.bfloat16, True, 7, False, 0, 0),
    ((5, 0, 33, 2), 96, 1, 128, torch.bfloat16, False, 0, False, 1, 0),
    ((40, 3), 64, 1, 64, torch.float32, True, 0, False, 0, 0),
    (EDGES, 4, 2, 128, torch.bfloat16, True, 2 ** 32 + 5, False, 0, 0),  # a window past every length
    ((1,), 1, 1, 64, torch.bfloat16, True, 0, False, 0, 0),
    ((1,), 1, 1, 8, torch.float32, True, 0, False, 0, 0),
    ((2500,), 4, 2, 128, torch.bfloat16, True, 0, False, 0, 0),
    ((2500, 1300), 2, 2, 256, torch.bfloat16, True, 700, False, 0, 0),
    ((2049,), 2, 1, 64, torch.bfloat16, False, 0, False, 0, 0),
    (tuple((53 * i) % 40 for i in range(300)), 4, 2, 128, torch.bfloat16, True, 0, False, 0, 0),
    (tuple(1 for i in range(1500)), 2, 1, 64, torch.bfloat16, True, 0, False, 0, 0),
    (tuple((53 * i) % 40 for i in range(100)), 4, 2, 64, torch.float32, True, 9, False, 0, 7),
    # long prompts in small batches: their keys split over a CTA's two query tiles
    ((257,), 2, 1, 128, torch.bfloat16, True, 0, False, 0, 0),
    ((481, 1, 640), 4, 2, 128, torch.bfloat16, True, 0, True, 5, 9),
    ((1000, 7, 399), 4, 4, 128, torch.bfloat16, False, 0, False, 0, 0),
    ((1601, 129), 2, 2, 128, torch.bfloat16, True, 450, False, 0, 3),
    ((385, 900), 4, 2, 64, torch.bfloat16, True, 0, True, 1, 1),
    ((1025, 513), 6, 2, 64, torch.bfloat16, False, 600, False, 0, 0),
    ((700,), 16, 1, 64, torch.bfloat16, True, 0, False, 0, 0),
    # more tiles than CTAs: no splits
    (EDGES + (600,), 64, 64, 128, torch.bfloat16, True, 0, False, 2, 2),
    (EDGES + (600,), 64, 64, 64, torch.bfloat16, True, 0, True, 0, 0),
    (EDGES + (600,), 64, 64, 64, torch.bfloat16, False, 200, False, 0, 0),
    (EDGES + (600,), 128, 64, 128, torch.bfloat16, True, 300, False, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{len(c[0])}max{max(c[0])}_h{c[1]}-{c[2]}_d{c[3]}_{str(c[4])[6:]}_c{int(c[5])}_w{c[6]}_f{int(c[7])}_{c[8]}-{c[9]}")
def test_packed_prefill_matches_the_definition(case):
    lens, Hq, Hkv, D, dtype, causal, window, fused, before, behind = case
    q, k, v, cu = make(lens, Hq, Hkv, D, dtype, fused, before, behind)
    scale = 1.0 / math.sqrt(D)
    y = run(q, k, v, cu, scale, causal, window)
    ref, tol = reference(q, k, v, cu, scale, causal, window)
    check(y, ref, tol, "y")  # rows outside every sequence: 7.0 as before, bound 0
    assert torch.equal(y, run(q, k, v, cu, scale, causal, window))


@pytest.mark.parametrize("D", [64, 128, 256, 96])
def test_other_sequences_never_reach_a_result(D):
    """NaN and infinities in one sequence's rows leave its neighbours' bits alone."""
    lens = (100, 60, 140, 33)
    q, k, v, cu = make(lens, 4, 2, D, torch.bfloat16)
    good = run(q, k, v, cu, 0.1, True, 0)
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2, q2 = k.clone(), v.clone(), q.clone()
        for t in (k2, v2, q2):
            t[100:160] = bad
        y = torch.full_like(good, 7.0)
        ek.attention_packed_prefill(y, q2, k2, v2, cu, 0.1)
        assert torch.equal(y[:100], good[:100]) and torch.equal(y[160:], good[160:])


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (256, torch.bfloat16), (64, torch.float32)])
def test_extreme_scores(D, dtype):
    """Peaked rows whose maximum keeps growing along the keys (every tile rescales), and equal keys."""
    n = 700
    q, k, v, cu = make((n,), 2, 1, D, dtype, sigma=1.0)
    k[:] = 0
    k[:, :, 0] = (torch.arange(n, device="cuda")[:, None] / 8).to(dtype)
    q[:, :, 0] = 8.0
    y = run(q, k, v, cu, 0.5, True, 0)
    ref, tol = reference(q, k, v, cu, 0.5, True, 0)
    check(y, ref, tol, "growing")
    q[:, :, 0] = -8.0
    y = run(q, k, v, cu, 0.5, True, 0)
    ref, tol = reference(q, k, v, cu, 0.5, True, 0)
    check(y, ref, tol, "falling")
    q.zero_()
    y = run(q, k, v, cu, 0.5, True, 0)
    ref, tol = reference(q, k, v, cu, 0.5, True, 0)
    check(y, ref, tol, "equal")


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float32)])
def test_bad_cu_seqlens_write_nothing(D, dtype):
    q, k, v, cu = make((40, 50, 10), 4, 2, D, dtype)
    for wrong in ([0, 40, 90, 101], [-1, 40, 90, 100], [0, 60, 40, 100], [0, 40, 1 << 40, 100], [100, 40, 90, 0]):
        y = torch.full_like(q, 7.0)
        st = ek.new_status()
        ek.attention_packed_prefill(y, q, k, v, torch.tensor(wrong, dtype=torch.int64, device="cuda"), 0.1, status=st)
        assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE and int(st[0]) == ek.EXTKV_DEV_BAD_SEQLENS
        assert (y == 7.0).all()
    y = run(q, k, v, cu, 0.1, True, 0)  # and a good call after them
    ref, tol = reference(q, k, v, cu, 0.1, True, 0)
    check(y, ref, tol, "after")


def test_other_stream_and_captured():
    lens = (300, 1, 0, 700)
    q, k, v, cu = make(lens, 8, 4, 128, torch.bfloat16)
    good = run(q, k, v, cu, 0.1, True, 0)
    s = torch.cuda.Stream()
    y = torch.zeros_like(good)
    s.wait_stream(torch.cuda.current_stream())
    ek.attention_packed_prefill(y, q, k, v, cu, 0.1, stream=s)
    s.synchronize()
    assert torch.equal(y, good)
    outs, graphs = [], []
    for _ in range(2):
        out = torch.zeros_like(good)
        call = ek.prepare_attention_packed_prefill(out, q, k, v, cu, 0.1, stream=s)
        call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        outs.append((out, call))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for out, _ in outs:
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for out, _ in outs:
        assert torch.equal(out, good)
    # the sequences' bounds may change between replays
    cu.copy_(torch.tensor([0, 10, 400, 401, 1001], device="cuda"))
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1][0], run(q, k, v, cu, 0.1, True, 0))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out_is_reported(D):
    """A poll limit of zero: the pipeline's waits give up, the status word says so,
    and the next call is whole again."""
    q, k, v, cu = make((300, 77), 4, 2, D, torch.bfloat16)
    y = torch.full_like(q, 7.0)
    st = ek.new_status()
    with ek.wait_polls(0):
        ek.attention_packed_prefill(y, q, k, v, cu, 0.1, status=st)
        assert "tcgen05" in ek.extkv_last_kernel()
    assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE and int(st[0]) == ek.EXTKV_DEV_TIMEOUT
    y = run(q, k, v, cu, 0.1, True, 0)
    ref, tol = reference(q, k, v, cu, 0.1, True, 0)
    check(y, ref, tol, "after")


@pytest.mark.parametrize("D,window", [(256, 90), (256, 0), (128, 90), (64, 0), (128, 0)])
def test_the_same_bits_from_cold_and_warm_caches(D, window):
    """Copies that land late, early and in other orders (L2 full of other data, or
    of this) change no bit."""
    lens = (1, 300, 129, 700, 64, 257)
    q, k, v, cu = make(lens, 8, 4, D, torch.bfloat16, True)
    other = torch.empty(1 << 26, dtype=torch.float32, device="cuda")  # twice the L2
    good = run(q, k, v, cu, 1.0 / math.sqrt(D), True, window)
    ref, tol = reference(q, k, v, cu, 1.0 / math.sqrt(D), True, window)
    check(good, ref, tol, "y")
    for i in range(60):
        if i % 3:
            other.fill_(float(i))
        if i % 3 == 2:
            k.sum()  # K warm, V cold
        assert torch.equal(run(q, k, v, cu, 1.0 / math.sqrt(D), True, window), good), i


def test_two_streams_at_once():
    """Calls with workspaces of their own, side by side on two streams."""
    sets = []
    for lens, Hq, Hkv, D in (((700, 1, 200), 16, 8, 256), ((900, 64), 8, 4, 128), ((500, 500), 4, 2, 64)):
        q, k, v, cu = make(lens, Hq, Hkv, D, torch.bfloat16)
        good = run(q, k, v, cu, 0.1, True, 0)
        s = torch.cuda.Stream()
        y = torch.zeros_like(good)
        sets.append((y, good, ek.prepare_attention_packed_prefill(y, q, k, v, cu, 0.1, stream=s)))
    torch.cuda.synchronize()
    for _ in range(10):
        for y, _, _ in sets:
            y.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for _, _, call in sets:
                call()
        torch.cuda.synchronize()
        for y, good, _ in sets:
            assert torch.equal(y, good)


def test_a_recorded_step():
    q, k, v, cu = make((100, 1, 300), 8, 2, 128, torch.bfloat16)
    good = run(q, k, v, cu, 0.1, True, 0)
    y = torch.zeros_like(good)
    ws = torch.empty(ek.attention_packed_prefill_workspace_size(q.shape[0], 3, 8, 2, 128, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    with ek.StepRecorder() as rec:
        ek.attention_packed_prefill(y, q, k, v, cu, 0.1, workspace=ws, stream=rec.stream)
    for _ in range(2):
        y.zero_()
        torch.cuda.synchronize()
        rec.step()
        torch.cuda.synchronize()
        assert torch.equal(y, good)
