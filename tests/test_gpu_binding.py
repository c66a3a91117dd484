"""The compiled binding writes each output into that tensor's own storage: a
lazy clone shares another tensor's until it is written, which stays as it was."""
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


class Outputs:
    """Tensors that a call is to write, each a lazy clone of one that is kept."""

    def __init__(self):
        self.kept, self.given = {}, {}

    def __call__(self, name, shape, dtype):
        base = torch.full(shape, 0x55, dtype=torch.uint8, device=G.DEV) if dtype == qb.F8 else \
            torch.full(shape, 85, dtype=dtype, device=G.DEV)
        base = base.view(qb.F8) if dtype == qb.F8 else base
        self.kept[name], self.given[name] = (base, base.clone()), torch._lazy_clone(base)
        return self.given[name]

    def check(self):
        torch.cuda.synchronize()
        bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
        for name, (base, was) in self.kept.items():
            assert torch.equal(bits(base), bits(was)), f"{name}: the tensor it was cloned from is overwritten"
            assert not torch.equal(bits(self.given[name]), bits(was)), f"{name}: nothing written"


def test_outputs_that_share_another_tensors_storage():
    N, E, K, H, M = 300, 32, 2, 64, 48
    g = torch.Generator(device=G.DEV).manual_seed(1)
    s, b = torch.rand((N, E), generator=g, device=G.DEV), torch.zeros(E, device=G.DEV)
    f32, i32, u8, bf16 = torch.float32, torch.int32, torch.uint8, torch.bfloat16
    new = Outputs()
    topk, gate = new("topk", (N, K), i32), new("gate", (N, K), f32)
    G.say("outputs as lazy clones")
    weight = new("weight", (1, E), f32)
    qb.qb_balance_forward(s, b, K, topk, gate=gate, count=new("count", (1, E), i32), weight=weight,
                          loss=new("loss", (1,), f32), ws=new("ws", (qb.qb_balance_workspace_bytes(N, E, 1),), u8),
                          coef=0.1)
    qb.qb_balance_backward(s, topk, weight=weight, dlogits=new("dlogits", (N, E), f32))
    R = qb.qb_dispatch_rows(N, K, E, 128)
    off, src, pos = new("off", (E + 1,), i32), new("row_src", (R,), i32), new("pos", (N, K), i32)
    qb.qb_dispatch(topk, E, 128, off, src, pos)
    rows, dout = torch.randn((R, H), generator=g, device=G.DEV).to(bf16), torch.randn((N, H), device=G.DEV).to(bf16)
    qb.qb_combine(rows, pos, new("out", (N, H), bf16), gate=gate)
    qb.qb_combine_backward(dout, rows, pos, src, new("drows", (R, H), bf16), gate=gate, dgate=new("dgate", (N, K), f32))
    xq, xs = new("xq", (R, qb.fp8_ld(H)), qb.F8), new("xs", (R, qb.fp8_sld(H)), u8)
    xt, xts = new("xt", (H, qb.fp8_ld(R)), qb.F8), new("xts", (H, qb.fp8_sld(R)), u8)
    qb.qb_fp8_quantize(dout, xq, xs, row_src=src)
    qb.qb_fp8_quantize_cols(dout, xt, xts, row_src=src)
    wq, ws = new("wq", (E, M, qb.fp8_ld(H)), qb.F8), new("w_scale", (E, 1, qb.fp8_sld(H)), u8)
    qb.qb_fp8_quantize_weight(torch.randn((E, M, H), generator=g, device=G.DEV), wq, ws,
                              new("wt", (E, H, qb.fp8_ld(M)), qb.F8), new("wts", (E, 1, qb.fp8_sld(M)), u8))
    qb.qb_fp8_product(xq, xs, wq, ws, new("y", (R, M), bf16), off=off)
    qb.qb_fp8_weight_grad(xt, xts, xt, xts, new("dw", (E, H, H), f32), off=off)
    new.check()
