"""How an expert layer takes its matrices, on the host alone: held in bfloat16
they are copied by torch, on whatever device they are."""
import torch

from exact_quantile_selection_amd.expert_layer import ExpertLayer


def test_matrices_that_an_optimizer_trains():
    """A parameter's copy is no step of its graph: the layer's products are not
    recorded, and each load would keep the one before."""
    w = torch.nn.Parameter(torch.randn((32, 16, 64)))
    layer = ExpertLayer(torch.zeros((32, 64), dtype=torch.bfloat16), w, 2, 10, held="bf16")
    for _ in range(2):
        assert not layer.w.requires_grad and layer.w.grad_fn is None
        assert torch.equal(layer.w, w.detach().to(torch.bfloat16))
        with torch.no_grad():
            w.mul_(0.5)
        layer.load_weights(w)
