"""The packed and paged operators write their outputs and nothing else: every
output, the pools, an exactly sized workspace and the status word are views into
larger allocations whose guard regions hold a byte pattern and must come back
whole; rows that belong to no sequence, and pool rows that no new row names, keep
their bits.  Inputs lie between guards that read as NaN, so that a row read past
an end would show in the result."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check, pages_for, rotary_bound, rotate_rows
from test_gpu_canaries import GUARD, PATTERN, Guarded
import test_gpu_packed_prefill as packed
import test_gpu_paged_decode as paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def between_nans(t):
    """A copy of t whose allocation goes on with NaN (floats) or far numbers (integers) on both sides."""
    pad = GUARD // t.element_size()
    bad = float("nan") if t.dtype.is_floating_point else (1 << 40)
    raw = torch.full((2 * pad + t.numel(),), bad, dtype=t.dtype, device="cuda")
    raw[pad:pad + t.numel()] = t.flatten()
    return raw[pad:pad + t.numel()].view(t.shape)


def guarded_status():
    st = Guarded((4,), torch.int32)
    st.view.zero_()
    return st


def intact(**guards):
    for name, g in guards.items():
        assert g.guards_intact(), f"{ek.extkv_last_kernel()} wrote outside {name}"


LENS = (0, 1, 17, 257, 3000)
DECODE = [(16, 8, 256, 16, 0, torch.bfloat16), (32, 2, 128, 64, 100, torch.bfloat16), (3, 1, 64, 48, 0, torch.bfloat16),
          (17, 1, 512, 32, 0, torch.bfloat16), (6, 2, 128, 7, 0, torch.bfloat16), (4, 2, 96, 16, 50, torch.bfloat16),
          (9, 1, 128, 24, 0, torch.float32)]


@pytest.mark.parametrize("algo", [ek.ALGO_DECODE_STREAMK, ek.ALGO_AUTO], ids=["axis", "auto"])
@pytest.mark.parametrize("window_lens", [LENS, (33,), tuple((37 * i) % 90 for i in range(200))], ids=["mix", "one", "many"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"h{c[0]}-{c[1]}_d{c[2]}_p{c[3]}_w{c[4]}_{str(c[5])[6:]}")
def test_paged_decode(case, window_lens, algo):
    Hq, Hkv, D, page, window, dtype = case
    lens, scale = window_lens, 1.0 / math.sqrt(D)
    q, k, v, table, nonpad = paged.make(lens, Hq, Hkv, D, page, dtype, window=window)
    qg, kg, vg, tg, ng = (between_nans(t) for t in (q, k, v, table, nonpad))
    y = Guarded((len(lens), Hq, D), dtype)
    ws = Guarded((ek.attention_paged_decode_workspace_size(len(lens), Hq, Hkv, D, dtype),), torch.uint8)
    st = guarded_status()
    with ek.use_algo(algo):
        ek.attention_paged_decode(y.view, qg, kg, vg, tg, ng, scale, window=window, workspace=ws.view, status=st.view)
    assert ek.extkv_read_status(st.view) == ek.EXTKV_OK, ek.extkv_last_error()
    intact(y=y, workspace=ws, status=st)
    ref, tol = paged.reference(q, k, v, table, lens, window, scale)
    check(y.view, ref, tol, "y")


@pytest.mark.parametrize("lens,before,behind", [((1, 0, 129, 300), 3, 5), ((2047,), 0, 0), ((20,), 0, 1), ((0, 0), 4, 4)],
                         ids=["mix", "split", "short", "none"])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 4, 128, torch.bfloat16), (6, 2, 64, torch.bfloat16), (4, 2, 256, torch.bfloat16),
                                            (4, 2, 96, torch.bfloat16), (4, 1, 512, torch.bfloat16), (6, 2, 128, torch.float32)],
                         ids=lambda x: str(x))
def test_packed_prefill(Hq, Hkv, D, dtype, lens, before, behind):
    scale = 1.0 / math.sqrt(D)
    if max(lens) > 1000 and not packed.fast(D, dtype):
        lens = (200,)
    q, k, v, cu = packed.make(lens, Hq, Hkv, D, dtype, False, before, behind)
    qg, kg, vg, cg = (between_nans(t) for t in (q, k, v, cu))
    y = Guarded(q.shape, dtype)
    y.view.fill_(7.0)
    ws = Guarded((ek.attention_packed_prefill_workspace_size(q.shape[0], len(lens), Hq, Hkv, D, dtype),), torch.uint8)
    st = guarded_status()
    ek.attention_packed_prefill(y.view, qg, kg, vg, cg, scale, workspace=ws.view, status=st.view)
    assert ek.extkv_read_status(st.view) == ek.EXTKV_OK, ek.extkv_last_error()
    intact(y=y, workspace=ws, status=st)
    ref, tol = packed.reference(q, k, v, cu, scale, True, 0)
    check(y.view, ref, tol, "y")
    if before:
        assert bool((y.view[:before] == 7.0).all())
    if behind:
        assert bool((y.view[-behind:] == 7.0).all())


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,R,inter,dtype", [
    ((5, 0, 300, 1), 8, 2, 64, 16, 64, False, torch.bfloat16), ((1,) * 9, 16, 8, 256, 16, 256, False, torch.bfloat16),
    ((5, 0, 30, 1), 4, 2, 128, 7, 96, True, torch.float32), ((5, 0, 30, 1), 3, 1, 8, 16, 6, False, torch.bfloat16),
    ((700, 3), 4, 2, 512, 32, 0, False, torch.bfloat16)], ids=lambda x: str(x))
def test_paged_append(lens, Hq, Hkv, D, page, R, inter, dtype):
    gen = torch.Generator().manual_seed(9)
    T, past, spare = sum(lens), 21, 4  # rows behind the last sequence
    pool, table = pages_for([n + past for n in lens], page, gen)
    x = torch.randn((T + spare, Hq + 2 * Hkv, D), generator=gen).to(dtype)
    q, kn, vn = (between_nans(t.contiguous()) for t in (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]))
    pools, old = [], []
    for _ in range(2):
        g = Guarded((pool, Hkv, page, D), dtype)
        g.view.copy_(torch.randn((pool, Hkv, page, D), generator=gen).to(dtype))
        pools.append(g)
        old.append(g.view.cpu())
    q_out, st = Guarded(q.shape, dtype), guarded_status()
    q_out.view.fill_(7.0)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()])
    pos = torch.randint(0, 10 ** 6, (1, T + spare), generator=gen)
    inv = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / max(1, R // 2)).float()
    rot = ek.RotarySpec(between_nans(pos), between_nans(inv), (R // 2,), inter) if R else None
    ek.paged_kv_append(pools[0].view, pools[1].view, kn, vn, between_nans(table),
                       between_nans(torch.full((len(lens),), past)), cu_seqlens=between_nans(cu), rotary=rot,
                       q_out=q_out.view if R else None, q=q if R else None, status=st.view)
    assert ek.extkv_read_status(st.view) == ek.EXTKV_OK, ek.extkv_last_error()
    intact(k_pages=pools[0], v_pages=pools[1], q_out=q_out, status=st)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).long()
    slot = past + torch.arange(T) - cu[seq]
    at = table[seq, slot // page], slice(None), slot % page
    for g, was, new in zip(pools, old, (kn, vn)):
        now = g.view.cpu()
        rows = now[at].clone()
        now[at] = was[at]
        assert torch.equal(now, was)  # nothing else moved
        if R and new is kn:
            ref, size = rotate_rows(new[:T], pos[:, :T], inv, (R // 2,), R, inter)
            check(rows, ref, rotary_bound(ref, size, dtype), "k")
        else:
            assert torch.equal(rows, new[:T].cpu())
    if R:
        ref, size = rotate_rows(q[:T], pos[:, :T], inv, (R // 2,), R, inter)
        check(q_out.view[:T].cpu(), ref, rotary_bound(ref, size, dtype), "q")
    assert bool((q_out.view[T if R else 0:] == 7.0).all())


@pytest.mark.parametrize("B,S,Hq,Hkv,D,R,inter,dtype", [
    (2, 33, 8, 2, 64, 64, False, torch.bfloat16), (1, 1, 16, 8, 256, 192, False, torch.bfloat16),
    (3, 5, 4, 1, 128, 30, True, torch.float32), (1, 700, 3, 1, 24, 10, False, torch.bfloat16)], ids=lambda x: str(x))
def test_rotary(B, S, Hq, Hkv, D, R, inter, dtype):
    gen = torch.Generator().manual_seed(10)
    pos = torch.randint(0, 10 ** 6, (1, B, S), generator=gen)
    inv = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2)).float()
    src = [torch.randn((B, H, S, D), generator=gen).to(dtype) for H in (Hq, Hkv)]
    out = [Guarded(t.shape, dtype) for t in src]
    ek.rotary_multi_axis(out[0].view, out[1].view, between_nans(src[0]), between_nans(src[1]),
                         ek.RotarySpec(between_nans(pos), between_nans(inv), (R // 2,), inter))
    intact(q_out=out[0], k_out=out[1])
    for g, t in zip(out, src):
        rows = t.transpose(1, 2).reshape(B * S, -1, D)
        ref, size = rotate_rows(rows, pos.view(1, -1), inv, (R // 2,), R, inter)
        got = g.view.cpu().transpose(1, 2).reshape(B * S, -1, D)
        check(got, ref, rotary_bound(ref, size, dtype), "rotary")


def test_the_guards_notice_a_write():
    g = Guarded((16,), torch.float32)
    assert g.guards_intact()
    g.raw[GUARD - 1] = PATTERN ^ 1
    assert not g.guards_intact()
