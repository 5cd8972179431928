"""The packed and paged operators on the library built with EXTKV_CHECKED, call
by call: no access outside its buffer, and the kinds of buffers that the call's
kernels address by computed indexes were all tested (status[3]; TMA copies need
no test), so that a clean status word means something.  Run as its own process
by tests/test_gpu_checked_buffers.py; prints "checked ok <calls>" at the end."""
import math
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import torch  # noqa: E402

from biased_gqa_attention_gb300 import build  # noqa: E402
from biased_gqa_attention_gb300 import extkv as ek  # noqa: E402

lib = ek.load(build.build(checked=True))
assert os.path.basename(lib._name) == "libextkv_checked.so", lib._name

import test_gpu_packed_prefill as prefill  # noqa: E402
import test_gpu_paged_decode as decode  # noqa: E402
from packed_ref import check, pages_for, rotary_bound, rotate_rows  # noqa: E402

LENS, TABLE, ROWS, PAGES, OUT, PARTIAL, ITEMS, ANGLES = (1 << i for i in range(8))  # common.cuh
B, F = torch.bfloat16, torch.float32
calls = 0


def done(st, kinds, what):
    global calls
    assert ek.extkv_read_status(st) == ek.EXTKV_OK, f"{what}: {ek.extkv_last_error()}"
    tested = int(st[3])
    assert tested == kinds, f"{what}: buffers tested {tested:#x}, not {kinds:#x}"
    calls += 1
    print(f"{what}: ok", flush=True)


AXIS, CLUSTER = ek.ALGO_DECODE_STREAMK, ek.ALGO_DECODE_CLUSTER
MMA = LENS | TABLE | ROWS | OUT
for lens, Hq, Hkv, D, page, window, dtype, algo, kinds in [
        ((5000, 3, 0, 257), 16, 8, 256, 16, 0, B, AXIS, MMA | PARTIAL),
        ((5000, 3, 0, 257), 32, 2, 128, 64, 300, B, AXIS, MMA | PARTIAL),
        ((5000, 3, 0, 257), 8, 4, 64, 16, 0, B, AXIS, MMA | PARTIAL),
        ((5000, 3, 0, 257), 17, 1, 512, 48, 0, B, AXIS, MMA | PARTIAL),
        ((5000, 3, 0, 257), 16, 8, 256, 16, 0, B, CLUSTER, MMA),
        ((5000, 3, 0, 257), 32, 2, 128, 64, 300, B, CLUSTER, MMA),
        ((5000, 3, 0, 257), 8, 4, 64, 16, 0, B, CLUSTER, MMA),
        ((5000, 3, 0, 257), 17, 1, 512, 48, 0, B, CLUSTER, MMA),
        ((1,), 2, 1, 64, 16, 0, B, AXIS, MMA | PARTIAL),
        (tuple((37 * i) % 90 for i in range(300)), 4, 2, 128, 16, 0, B, AXIS, MMA | PARTIAL),
        ((5000, 3, 0, 257), 6, 2, 128, 7, 0, B, AXIS, MMA | PARTIAL | PAGES),
        ((0, 1, 17, 257), 4, 2, 96, 16, 0, B, AXIS, MMA | PARTIAL | PAGES),
        ((0, 1, 17, 3000), 9, 1, 128, 24, 40, F, AXIS, MMA | PARTIAL | PAGES)]:
    q, k, v, table, nonpad = decode.make(lens, Hq, Hkv, D, page, dtype, window=window, q_gap=8)
    scale, st, y = 1 / math.sqrt(D), ek.new_status(), torch.zeros((len(lens), Hq, D), dtype=dtype, device="cuda")
    with ek.use_algo(algo):
        ek.attention_paged_decode(y, q, k, v, table, nonpad, scale, window=window, status=st)
    ref, tol = decode.reference(q, k, v, table, lens, window, scale)
    check(y, ref, tol, "decode")
    done(st, kinds, f"{ek.extkv_last_kernel()} D={D} page={page} {len(lens)} sequences")

TC = LENS | ITEMS | OUT
for lens, Hq, Hkv, D, dtype, window, kinds in [
        ((1, 0, 129, 300), 8, 4, 128, B, 0, TC), ((1, 0, 129, 300), 6, 2, 64, B, 90, TC), ((2047,), 8, 4, 128, B, 0, TC),
        ((1, 0, 129, 300), 4, 2, 256, B, 0, TC), ((1, 0, 129, 60), 4, 2, 96, B, 0, TC | ROWS),
        ((1, 0, 60), 4, 2, 512, B, 9, TC | ROWS), ((1, 0, 129, 60), 6, 2, 128, F, 20, TC | ROWS)]:
    q, k, v, cu = prefill.make(lens, Hq, Hkv, D, dtype, True, 3, 5)
    scale, st, y = 1 / math.sqrt(D), ek.new_status(), torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    ek.attention_packed_prefill(y, q, k, v, cu, scale, window=window, status=st)
    ref, tol = prefill.reference(q, k, v, cu, scale, True, window)
    check(y, ref, tol, "prefill")
    done(st, kinds, f"{ek.extkv_last_kernel()} D={D}")

for lens, with_cu, R, inter, dtype, Hq in [((5, 0, 300, 1), True, 64, False, B, 8), ((1,) * 9, False, 64, True, B, 8),
                                           ((5, 0, 30, 1), True, 48, False, F, 4), ((5, 0, 30, 1), True, 10, True, F, 4),
                                           ((5, 0, 30, 1), True, 0, False, B, 0)]:
    Hkv, D, page = 2, 64, 16
    gen = torch.Generator().manual_seed(5)
    T, past = sum(lens), 11
    pool, table = pages_for([n + past for n in lens], page, gen)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen).to(dtype).cuda()
    q, kn, vn = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    kp, vp = (torch.full((pool, Hkv, page, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()])
    at = torch.full((len(lens),), past, dtype=torch.int64, device="cuda")
    pos = torch.randint(0, 100000, (1, T), generator=gen)
    inv = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / max(R // 2, 1)).float()
    rot = ek.RotarySpec(pos.cuda(), inv.cuda(), (R // 2,), inter) if R else None
    st, q_out = ek.new_status(), torch.empty((T, Hq, D), dtype=dtype, device="cuda") if R else None
    ek.paged_kv_append(kp, vp, kn, vn, table.cuda(), at, cu_seqlens=cu.cuda() if with_cu else None, rotary=rot,
                       q_out=q_out, q=q if R else None, status=st)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).long()
    slot = past + torch.arange(T) - cu[seq]
    got_k, got_v = (p.cpu()[table[seq, slot // page], :, slot % page] for p in (kp, vp))
    assert torch.equal(got_v, vn.cpu())
    if R:
        for got, src in ((got_k, kn), (q_out.cpu(), q)):
            ref, size = rotate_rows(src, pos, inv, (R // 2,), R, inter)
            check(got, ref, rotary_bound(ref, size, dtype), "append")
    else:
        assert torch.equal(got_k, kn.cpu())
    done(st, LENS | TABLE | ROWS | PAGES | ((OUT | ANGLES) if R else 0), f"append R={R} {dtype}")
print(f"checked ok {calls}")
