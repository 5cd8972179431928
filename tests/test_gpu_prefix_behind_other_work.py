"""attention_shared_prefix_decode directly behind the kernels that make its inputs: rows appended and
queries turned by the append before it, lengths and tables changed on the stream, the same
buffers step after step, without a host between them and with one."""
import pytest
import torch

from biased_gqa_attention_gb300 import extkv as ek

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
STEPS = 48


@pytest.fixture(scope="module", autouse=True)
def _built():
    from biased_gqa_attention_gb300 import build
    build.build()


class Serving:
    """Sequences that grow by a token a step behind two prefixes whose pages change places every other step."""

    def __init__(self, B, Hq, Hkv, D, page, dtype, plen, wide):
        gen = torch.Generator(device="cuda").manual_seed(B)
        own, front = (STEPS + 20) // page + 2, plen // page + 1
        pool = B * own + 2 * front
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
        self.k, self.v = rand(pool, Hkv, page, D), rand(pool, Hkv, page, D)
        order = torch.randperm(pool, generator=torch.Generator().manual_seed(1)).cuda()
        self.table = order[:B * own].view(B, own).contiguous()
        self.front = torch.full((2, front + wide), -1, dtype=torch.int64, device="cuda")
        self.front[:, :front] = order[B * own:].view(2, front)
        self.plen = torch.tensor([plen, plen // 2], device="cuda")
        self.cu = torch.tensor([0, B // 2 + 1, B], device="cuda")
        self.nonpad = torch.arange(B, device="cuda") % 17
        self.widx = self.nonpad.clone()
        self.x = rand(STEPS, B, Hq + 2 * Hkv, D)
        self.q = torch.zeros((B, Hq, D), dtype=dtype, device="cuda")
        self.pos = torch.zeros((1, B), dtype=torch.int64, device="cuda")
        self.spec = ek.RotarySpec(self.pos, torch.rand(D // 2, generator=gen, device="cuda"), (D // 2,))
        self.y = torch.zeros((STEPS, B, Hq, D), dtype=dtype, device="cuda")
        self.ws = torch.full((ek.attention_shared_prefix_decode_workspace_size(B, 2, Hq, Hkv, D, dtype),), 0xFF, dtype=torch.uint8,
                             device="cuda")
        self.status = ek.new_status()
        self.Hq, self.Hkv = Hq, Hkv

    def run(self, between=lambda: None):
        Hq, Hkv = self.Hq, self.Hkv
        for i in range(STEPS):
            s = torch.cuda.current_stream()
            self.pos.add_(3)
            if i & 1:
                self.front.copy_(self.front.flip(0))
            self.nonpad.add_(1)
            between()
            x = self.x[i]
            ek.paged_kv_append(self.k, self.v, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], self.table, self.widx, rotary=self.spec,
                               q_out=self.q, q=x[:, :Hq], status=self.status, stream=s)
            between()
            ek.attention_shared_prefix_decode(self.y[i], self.q, self.k, self.v, self.front, self.plen, self.cu, self.table, self.nonpad,
                                              0.1, workspace=self.ws, status=self.status, stream=s)
            between()
            self.widx.add_(1)
        return self.y


CASES = [(6, 8, 2, 128, 16, BF, 300, 0, "shared_prefix_tcgen05"), (70, 8, 2, 128, 16, BF, 2000, 0, "shared_prefix_tcgen05_after"),
         (70, 8, 2, 128, 16, BF, 900, 0, "shared_prefix_tcgen05"),
         (70, 8, 2, 128, 64, BF, 2000, 16000, "shared_prefix_tcgen05_after"), (40, 4, 2, 64, 16, BF, 700, 0, "shared_prefix_tcgen05"),
         (12, 4, 2, 256, 16, BF, 700, 0, "shared_prefix_tcgen05"), (6, 4, 1, 512, 16, BF, 300, 0, "shared_prefix_simt_bf16"),
         (6, 4, 2, 64, 16, F32, 300, 0, "shared_prefix_simt_f32")]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c[0]}_h{c[1]}-{c[2]}_d{c[3]}_p{c[4]}_{str(c[5])[6:]}_P{c[6]}_w{c[7]}")
def test_steps_without_a_host_between(case):
    *shape, kernel = case
    want = Serving(*shape).run(torch.cuda.synchronize).clone()
    assert ek.extkv_last_kernel() == kernel
    assert bool(torch.isfinite(want.float()).all()) and bool(want.float().abs().amax((1, 2, 3)).gt(0).all())
    s = Serving(*shape)
    torch.cuda.synchronize()
    assert torch.equal(s.run(), want)
    assert ek.extkv_read_status(s.status) == ek.EXTKV_OK
    # recorded and replayed
    s = Serving(*shape)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.y, want)
    assert ek.extkv_read_status(s.status) == ek.EXTKV_OK
