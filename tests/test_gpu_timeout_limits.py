"""The prefill kernels when a pipeline wait gives up part of the way: under every
poll limit, from none to one that some waits meet, the call ends, is reported
when a wait gave up and is whole when none did, and the next call has the right
bits.  A wait that gives up leaves copies in flight; they land before the CTA
leaves, whichever warp gives up and when.  Nothing here faults, traps or hangs
the GPU: each wait is bounded and the kernels end by themselves."""
import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek
from biased_gqa_attention_gb300 import workloads as wl
from gpu_path import run_gpu, spec_of

SHORT = wl.Workload("limits_short", 331, B=2, Hq=8, Hkv=4, D=128, S_q=40, max_seq=256, dtype=torch.bfloat16,
                    causal=True, window=0, nonpad_range=(40, 100))
CASES = [(SHORT, "fused"), (SHORT, "bias"), (wl.small(wl.C5), "bias"), (wl.small(wl.C3), "fused")]


@pytest.mark.gpu
@pytest.mark.parametrize("w,mode", CASES, ids=lambda x: getattr(x, "name", str(x)))
def test_prefill_gives_up_cleanly(w, mode):
    inp = wl.make_inputs(w, "cuda")
    ref = run_gpu(inp, mode=mode, algo=ek.ALGO_PREFILL)
    y, st = torch.empty_like(ref["y"]), ek.new_status()
    kw = dict(bias=ref["bias"]) if mode == "bias" else dict(fused=spec_of(inp))
    gave_up = 0
    with ek.use_algo(ek.ALGO_PREFILL):
        for limit in (0, 1, 2, 7, 40, 150, 600):
            for _ in range(6):
                st.zero_()
                with ek.wait_polls(limit):
                    ek.attention_ext_kv(y, inp.q, ref["k"], ref["v"], inp.nonpad, w.scale, status=st, **kw)
                if ek.extkv_read_status(st) != ek.EXTKV_OK:
                    assert int(st[0]) == ek.EXTKV_DEV_TIMEOUT
                    gave_up += 1
                else:
                    assert torch.equal(y, ref["y"]), limit
                st.zero_()
                y.fill_(7.0)
                ek.attention_ext_kv(y, inp.q, ref["k"], ref["v"], inp.nonpad, w.scale, status=st, **kw)
                assert ek.extkv_read_status(st) == ek.EXTKV_OK, ek.extkv_last_error()
                assert torch.equal(y, ref["y"]), limit
    assert gave_up >= 6
