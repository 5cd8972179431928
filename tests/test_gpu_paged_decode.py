"""attention_paged_decode against the definition in 64 bits: lengths from zero
on, pages that end inside a tile, head groups of every kind, windows, garbage
(NaN) in every slot that is not live, few and many sequences."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import POISON, attention_rows, bound, check, pages_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def make(lens, Hq, Hkv, D, page, dtype, seed=0, window=0, q_gap=0, sigma=2.0):
    gen = torch.Generator().manual_seed(1234 + seed)
    pool, table = pages_for(lens, page, gen)
    kw = dict(generator=gen, dtype=torch.float32)
    B = len(lens)
    q = (torch.randn((B, Hq * D + q_gap), **kw) * sigma).to(dtype).cuda()[:, :Hq * D].view(B, Hq, D) if not q_gap else \
        (torch.randn((B, Hq * D + q_gap), **kw) * sigma).to(dtype).cuda().as_strided((B, Hq, D), (Hq * D + q_gap, D, 1))
    k = torch.randn((pool, Hkv, page, D), **kw).to(dtype)
    v = torch.randn((pool, Hkv, page, D), **kw).to(dtype)
    live = torch.zeros((pool, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window > 0 else 0
        j = torch.arange(lo, n)
        live[table[b, j // page], j % page] = True
    k[~live[:, None, :].expand(pool, Hkv, page)] = POISON
    v[~live[:, None, :].expand(pool, Hkv, page)] = POISON
    return q, k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int64).cuda()


def reference(q, k, v, table, lens, window, scale):
    B, Hq, D = q.shape
    Hkv, page = k.shape[1], k.shape[2]
    g = Hq // Hkv
    y = torch.zeros((B, Hq, D), dtype=torch.float64, device=q.device)
    tol = torch.full_like(y, 1e-30)
    p_bf16 = q.dtype == torch.bfloat16 and D in (64, 128, 256, 512)
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window > 0 else 0
        if n == lo:
            continue
        j = torch.arange(lo, n, device=q.device)
        at, off = table[b][j // page], j % page
        ok = torch.ones((g, n - lo), dtype=torch.bool, device=q.device)
        for h in range(Hkv):
            rows = slice(h * g, h * g + g)
            o, pv, size = attention_rows(q[b, rows], k[at, h, off], v[at, h, off], ok, scale)
            y[b, rows] = o
            tol[b, rows] = bound(o, pv, size, D, n - lo, q.dtype, p_bf16)
    return y, tol


def run(q, k, v, table, nonpad, scale, window, **kw):
    y = torch.full((q.shape[0], q.shape[1], q.shape[2]), 7.0, dtype=q.dtype, device=q.device)
    st = ek.new_status()
    ek.attention_paged_decode(y, q, k, v, table, nonpad, scale, window=window, status=st, **kw)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK, ek.extkv_last_error()
    return y


MIX = (0, 1, 15, 16, 17, 33, 257, 1000)
CASES = [
    # lens, Hq, Hkv, D, page, window, dtype
    (MIX, 16, 8, 256, 16, 0, torch.bfloat16),
    (MIX, 16, 8, 256, 16, 100, torch.bfloat16),
    (MIX, 8, 4, 128, 64, 0, torch.bfloat16),
    (MIX, 8, 8, 64, 32, 0, torch.bfloat16),
    (MIX, 16, 2, 512, 32, 0, torch.bfloat16),
    (MIX, 16, 2, 512, 32, 7, torch.bfloat16),
    (MIX, 32, 2, 128, 64, 0, torch.bfloat16),     # sixteen heads a unit
    (MIX, 24, 2, 256, 16, 300, torch.bfloat16),   # twelve
    (MIX, 20, 1, 64, 16, 0, torch.bfloat16),      # two row groups, the second of four heads
    (MIX, 17, 1, 512, 16, 0, torch.bfloat16),     # three groups of eight
    (MIX, 6, 2, 128, 7, 0, torch.bfloat16),       # three heads a KV head; pages end inside a tile
    (MIX, 5, 1, 128, 1, 0, torch.bfloat16),       # a page a slot
    (MIX, 4, 2, 128, 24, 20, torch.bfloat16),
    (MIX, 4, 2, 128, 4096, 0, torch.bfloat16),    # a page longer than the sequence
    (MIX, 4, 2, 96, 16, 0, torch.bfloat16),       # a head size without a tensor-core kernel
    (MIX, 4, 2, 8, 16, 0, torch.bfloat16),
    (MIX, 4, 2, 392, 16, 33, torch.bfloat16),
    (MIX, 4, 2, 64, 16, 0, torch.float32),
    (MIX, 22, 2, 128, 24, 0, torch.float32),
    (MIX, 4, 2, 200, 16, 100, torch.float32),
    (MIX, 9, 1, 512, 5, 0, torch.float32),
    (MIX, 128, 1, 64, 16, 2 ** 32 + 5, torch.bfloat16),   # a window past every length; eight row groups
    (MIX, 64, 1, 256, 48, 0, torch.bfloat16),     # a page of one and a half tiles of 32, three of 16
    (MIX, 2, 1, 64, 48, 50, torch.bfloat16),
    ((1,), 1, 1, 64, 16, 0, torch.bfloat16),
    ((1,), 1, 1, 8, 16, 0, torch.float32),
    ((20011,), 16, 8, 256, 16, 0, torch.bfloat16),          # one sequence over every slice
    ((20011, 3), 32, 2, 128, 64, 0, torch.bfloat16),
    ((9001,), 8, 2, 64, 16, 0, torch.float32),
    ((9001, 0, 40), 16, 2, 512, 32, 5000, torch.bfloat16),
    (tuple((37 * i) % 90 for i in range(700)), 4, 2, 128, 16, 0, torch.bfloat16),   # more sequences than a block's threads
    (tuple((37 * i) % 90 for i in range(400)), 4, 2, 64, 16, 0, torch.float32),
]


@pytest.mark.parametrize("algo", [ek.ALGO_AUTO, ek.ALGO_DECODE_STREAMK, ek.ALGO_DECODE_CLUSTER], ids=["auto", "axis", "cluster"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{len(c[0])}max{max(c[0])}_h{c[1]}-{c[2]}_d{c[3]}_p{c[4]}_w{c[5]}_{str(c[6])[6:]}")
def test_paged_decode_matches_the_definition(case, algo):
    lens, Hq, Hkv, D, page, window, dtype = case
    scale = 1.0 / math.sqrt(D)
    mma = dtype == torch.bfloat16 and D in (64, 128, 256, 512)
    q, k, v, table, nonpad = make(lens, Hq, Hkv, D, page, dtype, window=window)
    units = len(lens) * Hkv * -(-(Hq // Hkv) // (16 if Hq // Hkv > 8 and D <= 256 else 8))
    with ek.use_algo(algo):
        if algo == ek.ALGO_DECODE_CLUSTER and (not mma or page % 16 or units > 80):
            with pytest.raises(ek.ExtKVError) as e:
                run(q, k, v, table, nonpad, scale, window)
            assert e.value.code == ek.EXTKV_ERR_UNSUPPORTED
            return
        y = run(q, k, v, table, nonpad, scale, window)
        name = ek.extkv_last_kernel()
        # the same bits again, whatever the timing
        assert torch.equal(y, run(q, k, v, table, nonpad, scale, window))
    ref, tol = reference(q, k, v, table, lens, window, scale)
    check(y, ref, tol, "y")
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.count_nonzero(y[b]) == 0
    if not mma:
        assert name == f"paged_decode_simt_{'f32' if dtype == torch.float32 else 'bf16'}"
    else:
        assert name in {ek.ALGO_AUTO: ("paged_decode_mma", "paged_decode_cluster"), ek.ALGO_DECODE_STREAMK: ("paged_decode_mma",),
                        ek.ALGO_DECODE_CLUSTER: ("paged_decode_cluster",)}[algo]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_q_rows_may_be_strided(dtype):
    lens = (5, 300, 0, 64)
    q, k, v, table, nonpad = make(lens, 8, 4, 128, 16, dtype, q_gap=1024 + 8)
    assert q.stride(0) == 8 * 128 + 1032
    y = run(q, k, v, table, nonpad, 0.1, 0)
    assert torch.equal(y, run(q.contiguous(), k, v, table, nonpad, 0.1, 0))
    ref, tol = reference(q, k, v, table, lens, 0, 0.1)
    check(y, ref, tol, "y")


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_extreme_scores(dtype, D, each_kernel):
    """A peaked softmax (scores of hundreds), equal keys, and a key far above the rest."""
    lens = (400, 77)
    q, k, v, table, nonpad = make(lens, 4, 2, D, 16, dtype, sigma=40.0)
    y = run(q, k, v, table, nonpad, 1.0, 0)
    ref, tol = reference(q, k, v, table, lens, 0, 1.0)
    check(y, ref, tol, "peaked")
    q.zero_()  # every score 0: the mean of V
    y = run(q, k, v, table, nonpad, 1.0, 0)
    ref, tol = reference(q, k, v, table, lens, 0, 1.0)
    check(y, ref, tol, "equal")


@pytest.fixture(params=[ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO], ids=["axis", "auto"])
def each_kernel(request):
    with ek.use_algo(request.param):
        yield


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float32, 64), (torch.bfloat16, 512)])
def test_bad_lengths_and_pages_are_flagged_and_skipped(dtype, D, each_kernel):
    lens = (100, 40, 64, 200)
    q, k, v, table, nonpad = make(lens, 4, 2, D, 16, dtype)
    scale = 0.125
    good = run(q, k, v, table, nonpad, scale, 0)
    cap = table.shape[1] * 16
    for wrong in (-1, cap + 1, 1 << 40, -(1 << 62)):
        n2 = nonpad.clone()
        n2[1] = wrong
        y = torch.full_like(good, 7.0)
        st = ek.new_status()
        ek.attention_paged_decode(y, q, k, v, table, n2, scale, status=st)
        assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE
        assert int(st[0]) == ek.EXTKV_DEV_BAD_NONPAD and int(st[1]) == 1
        assert torch.count_nonzero(y[1]) == 0
        assert torch.allclose(y[[0, 2, 3]].float(), good[[0, 2, 3]].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    # a page outside the pool: its sixteen slots are skipped, the rest attended
    for wrong in (-1, k.shape[0], 1 << 50):
        t2 = table.clone()
        t2[3, 4] = wrong
        y = torch.full_like(good, 7.0)
        st = ek.new_status()
        ek.attention_paged_decode(y, q, k, v, t2, nonpad, scale, status=st)
        assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE
        assert int(st[0]) == ek.EXTKV_DEV_BAD_PAGE
        j = torch.tensor([x for x in range(200) if x // 16 != 4], device="cuda")
        at, off = table[3][j // 16], j % 16
        ok = torch.ones((2, len(j)), dtype=torch.bool, device="cuda")
        for h in range(2):
            o, pv, size = attention_rows(q[3, 2 * h:2 * h + 2], k[at, h, off], v[at, h, off], ok, scale)
            check(y[3, 2 * h:2 * h + 2], o, bound(o, pv, size, D, 200, dtype, dtype == torch.bfloat16), "rest")
    # every page of a sequence bad: a zero row
    t2 = table.clone()
    t2[2] = -5
    y = torch.full_like(good, 7.0)
    ek.attention_paged_decode(y, q, k, v, t2, nonpad, scale)
    assert torch.count_nonzero(y[2]) == 0 and torch.isfinite(y.float()).all()


@pytest.mark.parametrize("dtype,D,page", [(torch.bfloat16, 128, 7), (torch.float32, 64, 7), (torch.bfloat16, 128, 16)])
def test_a_bad_page_that_a_window_enters_midway_is_flagged(dtype, D, page, each_kernel):
    """The window's first key is neither a page's nor a tile's first row."""
    n, window = 100, 47
    q, k, v, table, nonpad = make((n,), 4, 2, D, page, dtype)
    lo = n - window
    assert lo % page and lo % 16
    table[0, lo // page] = -1
    y = torch.empty((1, 4, D), dtype=dtype, device="cuda")
    st = ek.new_status()
    ek.attention_paged_decode(y, q, k, v, table, nonpad, 0.1, window=window, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE and int(st[0]) == ek.EXTKV_DEV_BAD_PAGE
    good = make((n,), 4, 2, D, page, dtype)[3]
    j = torch.arange((lo // page + 1) * page, n, device="cuda")
    at, off = good[0][j // page], j % page
    ok = torch.ones((2, len(j)), dtype=torch.bool, device="cuda")
    p_bf16 = dtype == torch.bfloat16
    for h in range(2):
        o, pv, size = attention_rows(q[0, 2 * h:2 * h + 2], k[at, h, off], v[at, h, off], ok, 0.1)
        check(y[0, 2 * h:2 * h + 2], o, bound(o, pv, size, D, n, dtype, p_bf16), "rest")


def test_two_streams_at_once(each_kernel):
    """Calls with workspaces of their own, of both forms, side by side on two streams."""
    sets = []
    for i, (lens, Hq, Hkv, D) in enumerate((((517,), 16, 8, 256), ((4000, 300, 1, 77), 8, 2, 128))):
        q, k, v, table, nonpad = make(lens, Hq, Hkv, D, 16, torch.bfloat16, seed=i)
        good = run(q, k, v, table, nonpad, 0.1, 0)
        s = torch.cuda.Stream()
        y = torch.zeros_like(good)
        sets.append((y, good, ek.prepare_attention_paged_decode(y, q, k, v, table, nonpad, 0.1, stream=s)))
    torch.cuda.synchronize()
    for _ in range(10):
        for y, _, _ in sets:
            y.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for _, _, call in sets:
                call()
        torch.cuda.synchronize()
        for y, good, _ in sets:
            assert torch.equal(y, good)


def test_the_length_limits(each_kernel):
    """Full tables: every slot of every page live, lengths at the capacity."""
    for D, page, dtype in ((128, 16, torch.bfloat16), (256, 5, torch.bfloat16), (64, 16, torch.float32)):
        lens = (page * 9, page * 9)
        q, k, v, table, nonpad = make(lens, 4, 2, D, page, dtype)
        table = table[:, :9].contiguous()
        y = run(q, k, v, table, nonpad, 0.1, 0)
        ref, tol = reference(q, k, v, table, lens, 0, 0.1)
        check(y, ref, tol, "full")


def test_an_empty_table_and_an_empty_batch(each_kernel):
    q, k, v, table, nonpad = make((0, 0), 4, 2, 128, 16, torch.bfloat16)
    empty = table[:, :0].contiguous()
    y = run(q, k, v, empty, nonpad, 1.0, 0)
    assert torch.count_nonzero(y) == 0
    ek.attention_paged_decode(q[:0], q[:0], k, v, table[:0], nonpad[:0], 1.0)


def test_sequences_may_share_pages(each_kernel):
    """Two sequences with one prompt's pages in common."""
    lens = (200, 200)
    q, k, v, table, nonpad = make(lens, 8, 2, 128, 16, torch.bfloat16)
    table[1, :8] = table[0, :8]
    y = run(q, k, v, table, nonpad, 0.1, 0)
    ref, tol = reference(q, k, v, table, lens, 0, 0.1)
    check(y, ref, tol, "shared")


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes (and 2^31 elements) with the live pages at its end."""
    D, page, Hkv = 256, 64, 4
    pool = (1 << 31) // (page * Hkv * D) + 64
    k = torch.empty((pool, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in (k, v):
        t[-40:] = torch.randn((40, Hkv, page, D), generator=gen, device="cuda").to(torch.bfloat16)
        t[:8] = float("nan")
    lens = (1000, 130)
    table = torch.full((2, 17), -1, dtype=torch.int64, device="cuda")
    table[0, :16] = pool - 1 - torch.arange(16, device="cuda")
    table[1, :3] = pool - 20 - torch.arange(3, device="cuda")
    q = torch.randn((2, 8, D), generator=gen, device="cuda").to(torch.bfloat16)
    nonpad = torch.tensor(lens, dtype=torch.int64, device="cuda")
    y = run(q, k, v, table, nonpad, 0.06, 0)
    ref, tol = reference(q, k, v, table, lens, 0, 0.06)
    check(y, ref, tol, "far pages")


def test_other_stream_prepared_and_captured(each_kernel):
    lens = (300, 1, 0, 2000)
    q, k, v, table, nonpad = make(lens, 8, 4, 128, 16, torch.bfloat16)
    good = run(q, k, v, table, nonpad, 0.1, 0)
    s = torch.cuda.Stream()
    y = torch.zeros_like(good)
    s.wait_stream(torch.cuda.current_stream())
    ek.attention_paged_decode(y, q, k, v, table, nonpad, 0.1, stream=s)
    s.synchronize()
    assert torch.equal(y, good)
    # two captured graphs with a workspace each, replayed side by side
    outs, graphs = [], []
    for i in range(2):
        out = torch.zeros_like(good)
        with torch.cuda.stream(s):
            call = ek.prepare_attention_paged_decode(out, q, k, v, table, nonpad, 0.1, stream=s)
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
    # the lengths may change between replays
    nonpad.copy_(torch.tensor([17, 0, 0, 555], device="cuda"))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], run(q, k, v, table, nonpad, 0.1, 0))
    # a recorded step of the library
    out = torch.zeros_like(good)
    with ek.StepRecorder() as rec:
        call = ek.prepare_attention_paged_decode(out, q, k, v, table, nonpad, 0.1, workspace=torch.empty(
            ek.attention_paged_decode_workspace_size(4, 8, 4, 128, torch.bfloat16), dtype=torch.uint8, device="cuda"),
            stream=rec.stream)
        call()
    rec.step()
    torch.cuda.synchronize()
    assert torch.equal(out, outs[0][0])


@pytest.mark.parametrize("D,keys", [(64, 32), (128, 16), (256, 16), (512, 16)])
@pytest.mark.parametrize("per_warp", [1, 2, 5])
def test_one_sequence_over_every_warp(D, keys, per_warp):
    """Lengths that give every warp of the GPU about per_warp tiles: each CTA joins
    its warps' partials, the merge kernel the CTAs'."""
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 8
    n = warps * keys * per_warp + 3
    q, k, v, table, nonpad = make((n,), 4, 1, D, 64, torch.bfloat16)
    y = run(q, k, v, table, nonpad, 1.0 / math.sqrt(D), 0)
    ref, tol = reference(q, k, v, table, (n,), 0, 1.0 / math.sqrt(D))
    # the bound grows with the number of keys; the errors of independent roundings do not: hold the
    # result also to a tenth of one partial's share of the output
    check(y, ref, tol, "y")
    assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -7


def test_a_wait_that_runs_out_is_reported(each_kernel):
    """A poll limit of zero: the ring's waits give up, the status word says so, and
    the next call is whole again."""
    lens = (300, 77, 0, 5000)
    q, k, v, table, nonpad = make(lens, 4, 2, 128, 16, torch.bfloat16)
    y = torch.empty_like(q)
    st = ek.new_status()
    with ek.wait_polls(0):
        ek.attention_paged_decode(y, q, k, v, table, nonpad, 0.1, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE and int(st[0]) == ek.EXTKV_DEV_TIMEOUT
    y = run(q, k, v, table, nonpad, 0.1, 0)
    ref, tol = reference(q, k, v, table, lens, 0, 0.1)
    check(y, ref, tol, "after")


@pytest.mark.parametrize("D,g,page", [(64, 4, 16), (128, 2, 64), (128, 16, 16), (256, 2, 32), (512, 8, 16), (128, 3, 7), (96, 2, 16)])
def test_the_same_bits_from_cold_and_warm_caches(D, g, page, each_kernel):
    """Copies that land late, early and in other orders change no bit."""
    lens = (4000, 17, 900, 0, 2500, 333)
    q, k, v, table, nonpad = make(lens, 2 * g, 2, D, page, torch.bfloat16)
    other = torch.empty(1 << 26, dtype=torch.float32, device="cuda")  # twice the L2
    good = run(q, k, v, table, nonpad, 1.0 / math.sqrt(D), 0)
    for i in range(60):
        if i % 3:
            other.fill_(float(i))
        if i % 3 == 2:
            k.sum()  # K warm, V cold
        assert torch.equal(run(q, k, v, table, nonpad, 1.0 / math.sqrt(D), 0), good), i
