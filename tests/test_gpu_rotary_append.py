"""rotary_multi_axis and paged_kv_append against the definition with exact
angles, and the append's writes against a plain scatter, bit for bit."""
import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from packed_ref import check, pages_for, rotary_bound, rotate_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


def sections_of(half, axes):
    s = [half // axes] * axes
    s[-1] += half - sum(s)
    return tuple(s)


def inv_freq(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32)


ROTARY = [
    # B, S, Hq, Hkv, D, R, axes, interleaved, dtype, start
    (1, 1, 1, 1, 64, 64, 1, False, torch.bfloat16, 0),
    (2, 9, 4, 2, 128, 128, 3, False, torch.bfloat16, 5),
    (2, 9, 4, 2, 128, 96, 3, True, torch.bfloat16, 100000),
    (1, 5, 3, 1, 256, 192, 4, False, torch.bfloat16, 1 << 31),
    (3, 4, 2, 2, 64, 6, 2, False, torch.bfloat16, 77),      # a half of three pairs: single elements
    (3, 4, 2, 2, 64, 6, 2, True, torch.bfloat16, 77),
    (1, 7, 5, 1, 8, 2, 1, False, torch.bfloat16, 3),
    (1, 7, 5, 1, 4, 4, 1, True, torch.float32, 3),
    (2, 3, 4, 2, 64, 64, 1, True, torch.float32, 1 << 40),
    (2, 3, 4, 2, 512, 512, 3, False, torch.float32, -12345),
    (2, 3, 4, 2, 64, 10, 1, False, torch.float32, 9),
    (2, 700, 8, 4, 64, 64, 2, False, torch.bfloat16, 0),    # several rows a CTA
]


@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(str(x) for x in c).replace("torch.", ""))
def test_rotary_matches_the_definition(case):
    B, S, Hq, Hkv, D, R, axes, inter, dtype, start = case
    gen = torch.Generator().manual_seed(5)
    q = torch.randn((B, Hq, S, D), generator=gen).to(dtype).cuda()
    k = torch.randn((B, Hkv, S, D), generator=gen).to(dtype).cuda()
    pos = start + torch.randint(0, 5000, (axes, B, S), generator=gen)
    if start == 1 << 40:
        pos[0, 0, 0] = -(1 << 62)
        pos[0, 1, 1] = (1 << 63) - 1
    inv = inv_freq(R // 2)
    spec = ek.RotarySpec(pos.cuda(), inv.cuda(), sections_of(R // 2, axes), inter)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    ek.rotary_multi_axis(qo, ko, q, k, spec)
    rows = slice(0, None) if B * S < 100 else slice(0, None, 97)
    for x, o in ((q, qo), (k, ko)):
        flat = x.transpose(1, 2).reshape(B * S, x.shape[1], D)[rows]
        got = o.transpose(1, 2).reshape(B * S, x.shape[1], D)[rows].cpu()
        y, size = rotate_rows(flat, pos.reshape(axes, B * S)[:, rows], inv, spec.sections, R, inter)
        check(got, y, rotary_bound(y, size, dtype), "rotated")
        assert torch.equal(got[..., R:], flat[..., R:].cpu())
    # one tensor alone, and in place
    qa, ka = q.clone(), k.clone()
    ek.rotary_multi_axis(qa, None, qa, None, spec)
    ek.rotary_multi_axis(None, ka, None, ka, spec)
    assert torch.equal(qa, qo) and torch.equal(ka, ko)


def test_rotary_angles_far_out():
    """Position zero leaves bits alone; equal angles at any distance turn alike;
    a frequency that is not finite gives NaN in its pairs alone."""
    D = 64
    x = torch.randn((1, 1, 4, D), generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.zeros((1, 1, 4), dtype=torch.int64, device="cuda")
    inv = inv_freq(D // 2).cuda()
    o = torch.empty_like(x)
    ek.rotary_multi_axis(o, None, x, None, ek.RotarySpec(pos, inv, (D // 2,)))
    assert torch.equal(o, x)
    inv2 = inv.clone()
    inv2[3] = float("inf")
    inv2[5] = float("nan")
    ek.rotary_multi_axis(o, None, x, None, ek.RotarySpec(pos, inv2, (D // 2,)))
    bad = torch.isnan(o[0, 0, 0])
    assert bad.nonzero().flatten().tolist() == [3, 5, 35, 37]


def append_inputs(lens, starts, Hq, Hkv, D, page, dtype, gen, gap=0):
    T = sum(lens)
    pool, table = pages_for([s + n for s, n in zip(starts, lens)], page, gen)
    x = torch.randn((T, (Hq + 2 * Hkv) * D + gap), generator=gen).to(dtype).cuda()
    part = lambda h0, h: x[:, h0 * D:(h0 + h) * D].unflatten(1, (h, D))  # noqa: E731
    q, k, v = part(0, Hq), part(Hq, Hkv), part(Hq + Hkv, Hkv)
    kp = torch.randn((pool, Hkv, page, D), generator=gen).to(dtype).cuda()
    vp = torch.randn((pool, Hkv, page, D), generator=gen).to(dtype).cuda()
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64).cuda()
    return q, k, v, kp, vp, table.cuda(), torch.tensor(starts, dtype=torch.int64).cuda(), cu


def scatter_plain(pool, rows, table, starts, lens, page):
    out, t = pool.clone(), 0
    for b, n in enumerate(lens):
        slot = starts[b] + torch.arange(n, device=pool.device)
        out[table[b][slot // page], :, slot % page] = rows[t:t + n]
        t += n
    return out


APPEND = [
    # lens, starts, Hq, Hkv, D, page, R, axes, interleaved, dtype
    ((1,), (0,), 1, 1, 64, 16, 64, 1, False, torch.bfloat16),
    ((1, 1, 1, 1, 1), (0, 15, 16, 4000, 31), 16, 8, 256, 16, 256, 3, False, torch.bfloat16),
    ((5, 0, 33, 1), (3, 9, 0, 100), 8, 2, 128, 7, 96, 3, False, torch.bfloat16),
    ((5, 0, 33, 1), (3, 9, 0, 100), 8, 2, 128, 64, 128, 2, True, torch.bfloat16),
    ((20, 17), (0, 1), 4, 4, 64, 1, 6, 1, False, torch.float32),
    ((20, 17), (0, 1), 4, 2, 512, 24, 512, 4, True, torch.float32),
    ((900, 1201), (0, 55), 32, 2, 128, 64, 128, 3, False, torch.bfloat16),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"T{sum(c[0])}_" + "-".join(str(x) for x in c[2:]).replace("torch.", ""))
def test_append_rotates_and_writes(case):
    lens, starts, Hq, Hkv, D, page, R, axes, inter, dtype = case
    gen = torch.Generator().manual_seed(9)
    q, k, v, kp, vp, table, widx, cu = append_inputs(lens, starts, Hq, Hkv, D, page, dtype, gen, gap=64)
    T = sum(lens)
    # plain: bit-exact copies
    k0, v0 = kp.clone(), vp.clone()
    st = ek.new_status()
    ek.paged_kv_append(k0, v0, k, v, table, widx, cu_seqlens=cu, status=st)
    assert torch.equal(k0, scatter_plain(kp, k, table, starts, lens, page))
    assert torch.equal(v0, scatter_plain(vp, v, table, starts, lens, page))
    # rotated: the bits of rotary_multi_axis, then the same writes
    pos = torch.randint(0, 100000, (axes, T), generator=gen)
    spec = ek.RotarySpec(pos.cuda(), inv_freq(R // 2).cuda(), sections_of(R // 2, axes), inter)
    spec4 = ek.RotarySpec(spec.positions[:, None], spec.inv_freq, spec.sections, inter)
    qr, kr = (torch.empty((1, h, T, D), dtype=dtype, device="cuda") for h in (Hq, Hkv))
    ek.rotary_multi_axis(qr, kr, q.transpose(0, 1).contiguous()[None], k.transpose(0, 1).contiguous()[None], spec4)
    k1, v1, qo = kp.clone(), vp.clone(), torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")
    ek.paged_kv_append(k1, v1, k, v, table, widx, cu_seqlens=cu, rotary=spec, q_out=qo, q=q, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK, ek.extkv_last_error()
    assert torch.equal(qo, qr[0].transpose(0, 1))
    assert torch.equal(k1, scatter_plain(kp, kr[0].transpose(0, 1), table, starts, lens, page))
    assert torch.equal(v1, v0)
    # K alone
    k2 = kp.clone()
    ek.paged_kv_append(k2, vp.clone(), k, v, table, widx, cu_seqlens=cu, rotary=spec)
    assert torch.equal(k2, k1)
    if all(n == 1 for n in lens):  # a decode step needs no cu_seqlens
        k3, v3 = kp.clone(), vp.clone()
        ek.paged_kv_append(k3, v3, k, v, table, widx, rotary=spec, q_out=qo, q=q)
        assert torch.equal(k3, k1) and torch.equal(v3, v1)
        qd = q.contiguous()
        ek.paged_kv_append(k3, v3, k, v, table, widx, rotary=spec, q_out=qd, q=qd)
        assert torch.equal(qd, qo)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_bad_places_are_flagged_and_skipped(dtype):
    lens, starts, page, D = (5, 8, 3), (10, 0, 30), 16, 64
    gen = torch.Generator().manual_seed(2)
    q, k, v, kp, vp, table, widx, cu = append_inputs(lens, starts, 4, 2, D, page, dtype, gen)
    cap = table.shape[1] * page
    want = scatter_plain(kp, k, table, starts, lens, page)
    first = torch.zeros((kp.shape[0], page), dtype=torch.bool)  # slots of sequence 1
    first[table[1, 0].cpu(), :8] = True
    keep = first[:, None, :, None].expand_as(kp.cpu()).cuda()
    for wrong in (-1, cap - 7, 1 << 62, -(1 << 62), (1 << 63) - 1):
        w2 = widx.clone()
        w2[1] = wrong
        k2, v2, st = kp.clone(), vp.clone(), ek.new_status()
        ek.paged_kv_append(k2, v2, k, v, table, w2, cu_seqlens=cu, status=st)
        assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE
        assert int(st[0]) == ek.EXTKV_DEV_BAD_WRITE_IDX and int(st[1]) == 1
        assert torch.equal(k2, torch.where(keep, kp, want))
    for wrong in (-1, kp.shape[0], 1 << 60):
        t2 = table.clone()
        t2[1, 0] = wrong
        k2, v2, st = kp.clone(), vp.clone(), ek.new_status()
        pos = torch.arange(16, device="cuda")[None]
        qo = torch.empty((16, 4, D), dtype=dtype, device="cuda")
        ek.paged_kv_append(k2, v2, k, v, t2, widx, cu_seqlens=cu, status=st)
        assert int(st[0]) == ek.EXTKV_DEV_BAD_PAGE and int(st[1]) == 8
        assert torch.equal(k2, torch.where(keep, kp, want))
        ek.paged_kv_append(k2, v2, k, v, t2, widx, cu_seqlens=cu, q_out=qo, q=q,
                           rotary=ek.RotarySpec(pos, inv_freq(32).cuda(), (32,)))
        assert torch.isfinite(qo.float()).all()  # every q row is rotated all the same
    # cu_seqlens that breaks its rules: flagged, and no slot of another place is touched
    owned = torch.zeros((kp.shape[0], page), dtype=torch.bool)
    for b in range(3):
        for pg in table[b].tolist():
            if pg >= 0:
                owned[pg] = True
    for wrong in ([0, 5, 13, 17], [0, 9, 4, 16], [-3, 5, 13, 16], [0, 5, 1 << 40, 16]):
        k2, v2, st = kp.clone(), vp.clone(), ek.new_status()
        ek.paged_kv_append(k2, v2, k, v, table, widx, status=st,
                           cu_seqlens=torch.tensor(wrong, dtype=torch.int64, device="cuda"))
        assert ek.extkv_read_status(st) == ek.EXTKV_ERR_DEVICE and int(st[0]) & ek.EXTKV_DEV_BAD_SEQLENS
        assert torch.equal(k2[~owned.cuda()[:, None, :].expand(k2.shape[:3])], kp[~owned.cuda()[:, None, :].expand(k2.shape[:3])])


def test_rows_outside_every_sequence_are_left():
    lens, starts, page, D = (4, 6), (0, 3), 8, 64
    gen = torch.Generator().manual_seed(4)
    q, k, v, kp, vp, table, widx, cu = append_inputs((4, 6, 3), (0, 3, 0), 4, 2, D, page, torch.bfloat16, gen)
    pos = torch.arange(13, device="cuda")[None]
    qo = torch.full((13, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k2, v2 = kp.clone(), vp.clone()
    st = ek.new_status()
    ek.paged_kv_append(k2, v2, k, v, table[:2].contiguous(), widx[:2].contiguous(), cu_seqlens=cu[:3].contiguous(),
                       rotary=ek.RotarySpec(pos, inv_freq(32).cuda(), (32,)), q_out=qo, q=q, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK
    assert (qo[10:] == 7.0).all() and not (qo[:10] == 7.0).all()
    assert torch.equal(v2, scatter_plain(vp, v[:10], table, starts, lens, page))


def test_append_captured_and_on_another_stream():
    lens, starts, page, D = (1, 1, 1), (4, 100, 0), 16, 128
    gen = torch.Generator().manual_seed(6)
    q, k, v, kp, vp, table, widx, cu = append_inputs(lens, starts, 8, 2, D, page, torch.bfloat16, gen)
    pos = widx[None].repeat(3, 1).contiguous()
    spec = ek.RotarySpec(pos, inv_freq(64).cuda(), (16, 24, 24))
    want_k, want_v, want_q = kp.clone(), vp.clone(), torch.empty((3, 8, D), dtype=torch.bfloat16, device="cuda")
    ek.paged_kv_append(want_k, want_v, k, v, table, widx, rotary=spec, q_out=want_q, q=q)
    got_k, got_v, got_q = kp.clone(), vp.clone(), torch.zeros_like(want_q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ek.paged_kv_append(got_k, got_v, k, v, table, widx, rotary=spec, q_out=got_q, q=q, stream=s)
    s.synchronize()
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v) and torch.equal(got_q, want_q)
    got_k.copy_(kp)
    got_v.copy_(vp)
    got_q.zero_()
    call = ek.prepare_paged_kv_append(got_k, got_v, k, v, table, widx, rotary=spec, q_out=got_q, q=q, stream=s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v) and torch.equal(got_q, want_q)
    # the slots may move between replays
    widx += 1
    pos += 1
    g.replay()
    ek.paged_kv_append(want_k, want_v, k, v, table, widx, rotary=spec, q_out=want_q, q=q)
    torch.cuda.synchronize()
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v) and torch.equal(got_q, want_q)


def test_thousands_of_heads():
    """More heads than one CTA numbers: every row and head still lands once."""
    T, H, D = 800, 65535, 8
    gen = torch.Generator(device="cuda").manual_seed(8)
    k, v = (torch.randint(-30000, 30000, (T, H, D), dtype=torch.int16, device="cuda", generator=gen).view(torch.bfloat16)
            for _ in range(2))
    kp, vp = (torch.zeros((T, H, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(T, device="cuda")[None].contiguous()
    cu = torch.tensor([0, T], dtype=torch.int64, device="cuda")
    st = ek.new_status()
    ek.paged_kv_append(kp, vp, k, v, table, torch.zeros(1, dtype=torch.int64, device="cuda"), cu_seqlens=cu, status=st)
    assert ek.extkv_read_status(st) == ek.EXTKV_OK
    assert torch.equal(kp[:, :, 0].view(torch.int16), k.view(torch.int16))
    assert torch.equal(vp[:, :, 0].view(torch.int16), v.view(torch.int16))
