"""What an ExpertLayer keeps between forward and backward: the caller's own
tensors, which backward reads again, so that one written in between is an
error and not a wrong gradient."""
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from test_gpu_expert_layer import make

pytestmark = pytest.mark.gpu
N, E, K, H, M = 200, 32, 4, 256, 256


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def inputs():
    off = torch.tensor([0, N], dtype=torch.int32, device=G.DEV)
    return off, torch.ones(N, dtype=torch.uint8, device=G.DEV)


@pytest.mark.parametrize("which", ["h", "seq_off", "valid"])
def test_an_input_written_before_backward(which):
    layer, h, dout = make(N, E, K, H, M, 1, 1)
    off, valid = inputs()
    G.say(f"{which} written between forward and backward")
    layer.forward(h, seq_off=off, valid=valid)
    layer.backward(dout)                               # as they were
    dict(h=h, seq_off=off, valid=valid)[which].zero_()
    with pytest.raises(RuntimeError, match=f"{which} was written"):
        layer.backward(dout)
    layer.forward(h, seq_off=off, valid=valid)
    layer.backward(dout)
    torch.cuda.synchronize()


def test_another_layers_output_as_input():
    """A layer's output is its own buffer: its next forward writes it."""
    first, h, dout = make(N, E, K, H, M, 1, 2)
    second, _, _ = make(N, E, K, H, M, 1, 3)
    G.say("a layer's output written between forward and backward")
    second.forward(first.forward(h))
    dx = second.backward(dout)[0]
    first.backward(dx)
    first.forward(h)
    with pytest.raises(RuntimeError, match="h was written"):
        second.backward(dout)
    second.forward(dx)
    second.backward(dout)                              # writes dx, which was its input
    with pytest.raises(RuntimeError, match="h was written"):
        second.backward(dout)
    torch.cuda.synchronize()


def test_backward_needs_a_forward():
    layer, h, dout = make(N, E, K, H, M, 1, 4)
    with pytest.raises(RuntimeError, match="forward"):
        layer.backward(dout)
    with pytest.raises(RuntimeError, match="forward"):
        layer.update_bias()


def test_inputs_that_count_no_writes():
    """Tensors made under inference_mode have no count to look at."""
    layer, h, dout = make(N, E, K, H, M, 1, 5)
    with torch.inference_mode():
        x = h.clone()
        G.say("inference tensors")
        a = layer.forward(x).clone()
        layer.backward(dout)
    assert torch.equal(a, layer.forward(h))
    layer.backward(dout)
    torch.cuda.synchronize()
