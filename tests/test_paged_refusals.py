"""What the packed and paged entry points refuse, on the host, before any launch
(CPU only: the pointers are never used)."""
import ctypes
import itertools

import pytest
import torch

from biased_gqa_attention_gb300 import build as B_
from biased_gqa_attention_gb300 import extkv as ek

P = ctypes.c_void_p
GOOD, ODD = P(0x10000), P(0x10002)
INVALID, UNSUPPORTED, OK = ek.EXTKV_ERR_INVALID_ARG, ek.EXTKV_ERR_UNSUPPORTED, ek.EXTKV_OK


@pytest.fixture(scope="module")
def lib():
    B_.build()
    return ek.load()


def spec(axes=1, sections=(32,), R=64, inter=0, pos=0x10000, inv=0x10000):
    return ek._Rotary(axes, (ctypes.c_int32 * 4)(*sections), R, inter, pos, inv)


def rotary(lib, q_out=GOOD, k_out=GOOD, q=GOOD, k=GOOD, rot=None, B=1, Hq=4, Hkv=2, S=3, D=64, dtype=ek.EXTKV_BF16):
    return lib.rotary_multi_axis(q_out, k_out, q, k, ctypes.byref(rot or spec()), B, Hq, Hkv, S, D, dtype, None)


def test_rotary_refusals(lib):
    assert rotary(lib, dtype=9) == INVALID
    assert rotary(lib, Hq=0) == INVALID
    assert rotary(lib, D=60) == UNSUPPORTED          # 120 bytes a row
    assert rotary(lib, D=520) == UNSUPPORTED
    assert rotary(lib, B=-1) == INVALID
    assert rotary(lib, S=1 << 40) == INVALID
    assert rotary(lib, B=1 << 20, S=1 << 20) == INVALID
    assert rotary(lib, q=None) == INVALID and rotary(lib, k_out=None) == INVALID
    assert rotary(lib, q=ODD) == INVALID
    for bad in (spec(axes=0), spec(axes=5), spec(R=63), spec(R=0), spec(R=66, sections=(33,)), spec(sections=(31,)),
                spec(axes=2, sections=(40, -8)), spec(pos=None), spec(inv=None), spec(pos=0x10004), spec(inv=0x10001)):
        assert rotary(lib, rot=bad) == INVALID
        assert "rotary_multi_axis" in ek.extkv_last_error()
    assert lib.rotary_multi_axis(GOOD, GOOD, GOOD, GOOD, None, 1, 4, 2, 3, 64, 1, None) == INVALID
    assert rotary(lib, B=0) == OK and rotary(lib, S=0) == OK
    assert rotary(lib, q=None, q_out=None, k=None, k_out=None) == OK


def append(lib, rot=None, **kw):
    a = dict(kp=GOOD, vp=GOOD, kn=GOOD, vn=GOOD, table=GOOD, widx=GOOD, cu=GOOD, q_out=None, q=None, T=5, B=2, Hq=4, Hkv=2,
             D=64, num_pages=8, page=16, max_pages=4, qs=256, ks=128, vs=128, dtype=ek.EXTKV_BF16, status=None)
    a.update(kw)
    return lib.paged_kv_append(a["kp"], a["vp"], a["kn"], a["vn"], a["table"], a["widx"], a["cu"], a["q_out"], a["q"],
                               None if rot is None else ctypes.byref(rot), a["T"], a["B"], a["Hq"], a["Hkv"], a["D"],
                               a["num_pages"], a["page"], a["max_pages"], a["qs"], a["ks"], a["vs"], a["dtype"],
                               a["status"], None)


def test_append_refusals(lib):
    assert append(lib, dtype=7) == INVALID
    assert append(lib, D=12) == UNSUPPORTED
    assert append(lib, T=-1) == INVALID and append(lib, B=1 << 40) == INVALID
    assert append(lib, cu=None) == INVALID           # five rows for two sequences
    assert "one row per sequence" in ek.extkv_last_error()
    assert append(lib, num_pages=0) == INVALID and append(lib, page=0) == INVALID and append(lib, max_pages=-1) == INVALID
    assert append(lib, num_pages=1 << 30, page=16) == UNSUPPORTED
    assert append(lib, max_pages=1 << 30) == UNSUPPORTED
    assert append(lib, q=GOOD) == INVALID and append(lib, q=GOOD, q_out=GOOD) == INVALID  # no rotary
    assert append(lib, rot=spec(), q=GOOD, q_out=GOOD, qs=264) == INVALID                 # in place, not dense
    assert append(lib, rot=spec(), q=GOOD, q_out=P(0x20000), qs=255) == INVALID
    assert append(lib, rot=spec(sections=(5,))) == INVALID
    assert append(lib, ks=127) == INVALID and append(lib, vs=132) == INVALID and append(lib, ks=64) == INVALID
    for name in ("kp", "vp", "kn", "vn", "table", "widx"):
        assert append(lib, **{name: None}) == INVALID, name
    for name in ("kp", "vp", "kn", "vn", "table", "widx", "cu", "status"):
        assert append(lib, **{name: ODD}) == INVALID, name
    assert append(lib, T=0) == OK and append(lib, B=0) == OK


def decode(lib, **kw):
    a = dict(y=GOOD, q=GOOD, kp=GOOD, vp=GOOD, table=GOOD, nonpad=GOOD, scale=1.0, window=0, B=2, Hq=4, Hkv=2, D=64,
             num_pages=8, page=16, max_pages=4, qs=256, dtype=ek.EXTKV_BF16, ws=GOOD, n=1 << 40, status=None)
    a.update(kw)
    return lib.attention_paged_decode(a["y"], a["q"], a["kp"], a["vp"], a["table"], a["nonpad"], a["scale"], a["window"],
                                      a["B"], a["Hq"], a["Hkv"], a["D"], a["num_pages"], a["page"], a["max_pages"], a["qs"],
                                      a["dtype"], a["ws"], a["n"], a["status"], None)


def prefill(lib, **kw):
    a = dict(y=GOOD, q=GOOD, k=GOOD, v=GOOD, cu=GOOD, scale=1.0, causal=1, window=0, T=9, B=2, Hq=4, Hkv=2, D=64, qs=256,
             ks=128, vs=128, dtype=ek.EXTKV_BF16, ws=GOOD, n=1 << 40, status=None)
    a.update(kw)
    return lib.attention_packed_prefill(a["y"], a["q"], a["k"], a["v"], a["cu"], a["scale"], a["causal"], a["window"], a["T"],
                                        a["B"], a["Hq"], a["Hkv"], a["D"], a["qs"], a["ks"], a["vs"], a["dtype"], a["ws"],
                                        a["n"], a["status"], None)


@pytest.mark.parametrize("call", [decode, prefill])
def test_attention_refusals(lib, call):
    assert call(lib, dtype=5) == INVALID
    assert call(lib, Hq=5) == INVALID and "multiple" in ek.extkv_last_error()
    assert call(lib, Hq=0) == INVALID and call(lib, Hkv=0) == INVALID and call(lib, B=-1) == INVALID
    assert call(lib, D=12) == UNSUPPORTED and call(lib, D=520) == UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, scale=scale) == INVALID
    assert call(lib, n=16) == INVALID and "workspace" in ek.extkv_last_error()
    assert call(lib, ws=None) == INVALID and call(lib, ws=P(0x10010)) == INVALID
    assert call(lib, qs=255) == INVALID and call(lib, qs=260) == INVALID and call(lib, qs=(1 << 33)) == INVALID
    for name in ("y", "q") + (("kp", "vp", "table", "nonpad") if call is decode else ("k", "v", "cu")):
        assert call(lib, **{name: None}) == INVALID, name
        assert call(lib, **{name: ODD}) == INVALID, name
    assert call(lib, status=ODD) == INVALID
    assert call(lib, B=0) == OK


def test_more_attention_refusals(lib):
    assert decode(lib, num_pages=0) == INVALID and decode(lib, page=-1) == INVALID
    assert decode(lib, max_pages=1 << 28) == UNSUPPORTED and decode(lib, num_pages=1 << 31) == UNSUPPORTED
    assert decode(lib, B=1 << 30) == INVALID
    assert prefill(lib, T=1 << 31) == UNSUPPORTED and prefill(lib, T=-1) == INVALID
    assert prefill(lib, ks=127) == INVALID and prefill(lib, vs=64) == INVALID
    assert prefill(lib, T=0) == OK
    assert lib.attention_paged_decode_workspace_size(0, 4, 2, 64, 1) == 0
    assert lib.attention_packed_prefill_workspace_size(9, 2, 5, 2, 64, 1) == 0
    for D, dt in itertools.product((8, 64, 128, 256, 512), (0, 1)):
        assert lib.attention_paged_decode_workspace_size(3, 8, 4, D, dt) > 0
        assert lib.attention_packed_prefill_workspace_size(100, 3, 8, 4, D, dt) > 0


def test_the_binding_checks_shapes_and_devices():
    f = torch.bfloat16
    q, y = torch.zeros((2, 4, 64), dtype=f), torch.zeros((2, 4, 64), dtype=f)
    kp = torch.zeros((8, 2, 16, 64), dtype=f)
    table, n = torch.zeros((2, 4), dtype=torch.int64), torch.zeros(2, dtype=torch.int64)
    call = ek.prepare_attention_paged_decode
    with pytest.raises(ValueError, match="CUDA"):
        call(y, q, kp, kp, table, n, 1.0, stream=0)
    with pytest.raises(ValueError):
        call(y, q, kp, kp, table[:1], n, 1.0, stream=0)
    with pytest.raises(ValueError):
        call(y, q, kp, kp[:4], table, n, 1.0, stream=0)
    with pytest.raises(ValueError):
        call(y[:, :2], q, kp, kp, table, n, 1.0, stream=0)
    with pytest.raises(TypeError):
        call(y, q, kp.float(), kp.float(), table, n, 1.0, stream=0)
    with pytest.raises(TypeError):
        call(y, q, kp, kp, table.int(), n, 1.0, stream=0)
    with pytest.raises(ValueError):  # heads that are not dense
        call(y, torch.zeros((2, 4, 128), dtype=f)[:, :, ::2], kp, kp, table, n, 1.0, stream=0)
    with pytest.raises(ValueError):
        call(y, q, kp, kp, table, n, 1.0, status=torch.zeros(2, dtype=torch.int32), stream=0)
    k = torch.zeros((2, 2, 64), dtype=f)
    cu = torch.tensor([0, 2])
    pre = ek.prepare_attention_packed_prefill
    with pytest.raises(ValueError, match="CUDA"):
        pre(y, q, k, k, cu, 1.0, stream=0)
    with pytest.raises(ValueError):
        pre(y, q, k, k[:1], cu, 1.0, stream=0)
    with pytest.raises(ValueError):
        pre(y, q, k, k, cu[:0], 1.0, stream=0)
    pos, inv = torch.zeros((1, 2), dtype=torch.int64), torch.ones(32)
    app = ek.prepare_paged_kv_append
    good = ek.RotarySpec(pos, inv, (32,))
    with pytest.raises(ValueError, match="CUDA"):
        app(kp, kp, k, k, table, n, rotary=good, stream=0)
    for bad in (ek.RotarySpec(pos, inv, (31,)), ek.RotarySpec(pos, inv, ()), ek.RotarySpec(pos[:, :1], inv, (32,)),
                ek.RotarySpec(pos, inv, (8, 8, 8, 4, 4))):
        with pytest.raises(ValueError):
            app(kp, kp, k, k, table, n, rotary=bad, stream=0)
    with pytest.raises(ValueError):
        app(kp, kp, k, k, table, n, q=q, q_out=y, stream=0)
    with pytest.raises(ValueError):
        app(kp, kp, k[:1], k[:1], table, n, stream=0)
    with pytest.raises(ValueError):
        app(kp, kp, k, k, table, n, cu_seqlens=cu, stream=0)
    x = torch.zeros((1, 4, 2, 64), dtype=f)
    rot = ek.prepare_rotary_multi_axis
    with pytest.raises(ValueError, match="CUDA"):
        rot(x, None, x, None, ek.RotarySpec(pos[:, None], inv, (32,)), stream=0)
    with pytest.raises(ValueError):
        rot(x, None, x, x, good, stream=0)
    with pytest.raises(ValueError):
        rot(None, None, None, None, good, stream=0)
