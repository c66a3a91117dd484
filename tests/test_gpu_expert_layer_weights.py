"""An expert layer's matrices between forward and backward: backward reads them
again, so that others laid out in between are an error and not a wrong gradient."""
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from test_gpu_expert_layer_held import make

pytestmark = pytest.mark.gpu
N, E, K, H, M = 200, 32, 4, 256, 96


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


@pytest.mark.parametrize("held", ["e4m3", "bf16", "e2m1"])
def test_matrices_laid_out_before_backward(held):
    layer, w, h, dout = make(N, E, K, H, M, held, 1)
    G.say(f"matrices laid out between forward and backward, held={held}")
    layer.forward(h)
    first = layer.backward(dout)[0].clone()
    assert torch.equal(layer.backward(dout)[0], first)  # as they were
    layer.load_weights(w * 2)
    with pytest.raises(RuntimeError, match="w was written"):
        layer.backward(dout)
    layer.load_weights(w)
    layer.forward(h)
    assert torch.equal(layer.backward(dout)[0], first)
    torch.cuda.synchronize()


@pytest.mark.parametrize("held", ["e4m3", "bf16", "e2m1"])
def test_a_layer_made_in_inference_mode(held):
    """Its buffers count no writes."""
    G.say(f"a layer made in inference mode, held={held}")
    with torch.inference_mode():
        layer, w, h, dout = make(N, E, K, H, M, held, 2)
        layer.load_weights(w)
        out = layer.forward(h).clone()
        dx = layer.backward(dout)[0].clone()
        layer.orthogonalized()
    other, _, _, _ = make(N, E, K, H, M, held, 2)
    other.b.copy_(layer.b)
    assert torch.equal(other.forward(h), out) and torch.equal(other.backward(dout)[0], dx)
    torch.cuda.synchronize()
