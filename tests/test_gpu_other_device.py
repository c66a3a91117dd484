"""The expert layer's calls run on the device that their tensors are on: a
stream of another one, or another current device, is refused before anything is
launched."""
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


def new(*shape, dtype=torch.bfloat16):
    return torch.ones(shape, dtype=dtype, device=G.DEV)


def calls():
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    x, w, y = new(4, 8), new(6, 8), new(4, 6)
    xq, xs, wq, ws = new(4, 128, dtype=u8), new(4, 8, dtype=u8), new(6, 128, dtype=u8), new(6, 8, dtype=u8)
    o, work = new(6, 8), new(qb.qb_orthogonalize_workspace_bytes(1, 6, 8), dtype=u8)
    pos, out, f, dw = torch.zeros((4, 2), dtype=i32, device=G.DEV), new(4, 8), new(6, 8, dtype=f32), new(6, 8, dtype=f32)
    return {
        "bf16_product": lambda **k: qb.qb_bf16_product(x, w, y, **k),
        "bf16_weight_grad": lambda **k: qb.qb_bf16_weight_grad(y, x, dw, **k),
        "fp4_quantize": lambda **k: qb.qb_fp4_quantize(x, xq, xs, **k),
        "fp4_quantize_weight": lambda **k: qb.qb_fp4_quantize_weight(f, wq, ws, **k),
        "fp4_product": lambda **k: qb.qb_fp4_product(xq, xs, wq, ws, y, **k),
        "orthogonalize": lambda **k: qb.qb_orthogonalize(f, o, work, **k),
        "combine": lambda **k: qb.qb_combine(x, pos, out, **k),
    }


class Stream:
    """A stream of a second device, as far as a call looks at it."""
    cuda_stream, device_index = 0, 1


@pytest.mark.parametrize("name", ["bf16_product", "bf16_weight_grad", "fp4_quantize", "fp4_quantize_weight", "fp4_product",
                                  "orthogonalize", "combine"])
def test_another_device(name, monkeypatch):
    call = calls()[name]
    G.say(f"{name} with another current device")
    call()
    call(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="tensors are on cuda:0, the stream is of cuda:1"):
        call(stream=Stream())
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        with pytest.raises(ValueError, match="tensors are on cuda:0, the current device is cuda:1"):
            call()
