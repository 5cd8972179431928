"""A prompt and the steps after it through the operators together: rotate and
write the prompt's rows into pages, attend the packed prompts, then token by
token rotate, write and attend over the pages, against the definition in 64
bits on the rows that the pages hold."""
import math

import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import attention_rows, bound, check, pages_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype,D,Hq,Hkv,page,window", [(torch.bfloat16, 128, 8, 4, 16, 0), (torch.bfloat16, 256, 16, 8, 32, 40),
                                                        (torch.float32, 64, 4, 2, 16, 0)])
def test_prompt_then_steps(dtype, D, Hq, Hkv, page, window):
    lens, steps = (37, 1, 130, 64), 3
    B, T, g, scale = len(lens), sum(lens), Hq // Hkv, 1 / math.sqrt(D)
    gen = torch.Generator().manual_seed(21)
    pool, table = pages_for([n + steps for n in lens], page, gen)
    table = table.cuda()
    kp = torch.full((pool, Hkv, page, D), float("nan"), dtype=dtype, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    inv = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    sections = (D // 2 - 2 * (D // 8), D // 8, D // 8)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64).cuda()
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=gen).to(dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.cat([torch.arange(n) for n in lens])[None].repeat(3, 1)
    pos[1] //= 8
    pos[2] %= 8
    st = ek.new_status()
    zero = torch.zeros(B, dtype=torch.int64, device="cuda")
    qr, y = torch.empty((T, Hq, D), dtype=dtype, device="cuda"), torch.empty((T, Hq, D), dtype=dtype, device="cuda")
    ek.paged_kv_append(kp, vp, k, v, table, zero, cu_seqlens=cu, rotary=ek.RotarySpec(pos.cuda(), inv, sections), q_out=qr,
                       q=q, status=st)
    # the rotated K rows, packed again from the pages
    rows = torch.cat([table[b, torch.arange(n, device="cuda") // page] for b, n in enumerate(lens)])
    offs = torch.cat([torch.arange(n, device="cuda") % page for n in lens])
    kr, vr = kp[rows, :, offs], vp[rows, :, offs]
    assert torch.equal(vr, v)
    ek.attention_packed_prefill(y, qr, kr, vr, cu, scale, window=window, status=st)
    t0 = 0
    for n in lens:
        i = torch.arange(n, device="cuda")
        ok = i[None] <= i[:, None]
        if window:
            ok &= i[:, None] - i[None] < window
        for h in range(Hq):
            o, pv, size = attention_rows(qr[t0:t0 + n, h], kr[t0:t0 + n, h // g], vr[t0:t0 + n, h // g], ok, scale)
            check(y[t0:t0 + n, h], o, bound(o, pv, size, D, n, dtype, dtype == torch.bfloat16), "prompt")
        t0 += n
    nonpad = torch.tensor(lens, dtype=torch.int64, device="cuda")
    for step in range(steps):
        x = torch.randn((B, Hq + 2 * Hkv, D), generator=gen).to(dtype).cuda()
        q1, k1, v1 = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        qs, ys = torch.empty((B, Hq, D), dtype=dtype, device="cuda"), torch.empty((B, Hq, D), dtype=dtype, device="cuda")
        spec = ek.RotarySpec(nonpad[None].repeat(3, 1).contiguous(), inv, sections)
        ek.paged_kv_append(kp, vp, k1, v1, table, nonpad, rotary=spec, q_out=qs, q=q1, status=st)
        nonpad += 1
        ek.attention_paged_decode(ys, qs, kp, vp, table, nonpad, scale, window=window, status=st)
        for b, n in enumerate(nonpad.tolist()):
            lo = max(0, n - window) if window else 0
            j = torch.arange(lo, n, device="cuda")
            at, off = table[b][j // page], j % page
            for h in range(Hkv):
                r = slice(h * g, h * g + g)
                ok = torch.ones((g, n - lo), dtype=torch.bool, device="cuda")
                o, pv, size = attention_rows(qs[b, r], kp[at, h, off], vp[at, h, off], ok, scale)
                check(ys[b, r], o, bound(o, pv, size, D, n, dtype, dtype == torch.bfloat16), f"step {step}")
    assert ek.extkv_read_status(st) == ek.EXTKV_OK, ek.extkv_last_error()


def test_a_decode_step_from_one_prompt_token_equals_the_prompts_last_row():
    """Attention of the last prompt row over packed rows and over pages: the two
    operators agree within both bounds."""
    n, Hq, Hkv, D, page = 333, 8, 2, 128, 16
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((n, h, D), generator=gen).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    pool, table = pages_for([n], page, gen)
    table = table.cuda()
    kp = torch.zeros((pool, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    cu = torch.tensor([0, n], dtype=torch.int64, device="cuda")
    ek.paged_kv_append(kp, vp, k, v, table, torch.zeros(1, dtype=torch.int64, device="cuda"), cu_seqlens=cu)
    y, y1 = torch.empty_like(q), torch.empty_like(q[-1:])
    ek.attention_packed_prefill(y, q, k, v, cu, 0.088)
    ek.attention_paged_decode(y1, q[-1:], kp, vp, table, torch.tensor([n], dtype=torch.int64, device="cuda"), 0.088)
    for h in range(Hq):
        ok = torch.ones((1, n), dtype=torch.bool, device="cuda")
        o, pv, size = attention_rows(q[-1:, h], k[:, h // 4], v[:, h // 4], ok, 0.088)
        b = bound(o, pv, size, D, n, torch.bfloat16, True)
        check(y[-1:, h], o, b, "prompt")
        check(y1[:, h], o, b, "step")
