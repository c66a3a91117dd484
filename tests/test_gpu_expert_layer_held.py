"""The expert layer with its matrices held in bfloat16 and in 4 bits: a training
step stage by stage against its definition in float64, from the values that the
stage before left, and an optimizer's step made of its own gradient.

Tolerances: a bf16 result is off by half a step, 2^-8 of it; a sum of n terms in
32 bits by n 2^-23 of their magnitudes.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb
from exact_quantile_selection_amd.expert_layer import ExpertLayer

import gpu_util as G
from test_gpu_expert_layer import close
from test_gpu_fp4 import values
from test_gpu_ortho import near as near_ortho

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def make(N, E, K, H, M, held, seed, B=1):
    g = torch.Generator(device=G.DEV).manual_seed(seed)
    wr = torch.randn((E, H), generator=g, device=G.DEV) / H ** 0.5
    w = torch.randn((E, M, H), generator=g, device=G.DEV) / H ** 0.5
    layer = ExpertLayer(wr.to(torch.bfloat16), w, K, N, coef=1e-2, B=B, held=held)
    layer.b.copy_((torch.rand(E, generator=g, device=G.DEV) - 0.5) * 0.1)
    h = torch.randn((N, H), generator=g, device=G.DEV).to(torch.bfloat16)
    dout = torch.randn((N, M), generator=g, device=G.DEV).to(torch.bfloat16)
    return layer, w, h, dout


def on_gpu(a):
    return torch.from_numpy(a).to(G.DEV)


@pytest.mark.parametrize("held", ["bf16", "e2m1"])
@pytest.mark.parametrize("N,E,K,H,M", [(300, 32, 2, 256, 200), (1000, 64, 6, 512, 130), (16, 256, 8, 256, 384),
                                       (2500, 32, 8, 384, 264)])
def test_a_training_step(N, E, K, H, M, held):
    layer, w, h, dout = make(N, E, K, H, M, held, N + E)
    valid = torch.ones(N, dtype=torch.uint8, device=G.DEV)
    valid[N // 2:N // 2 + 3] = 0
    h[N // 2:N // 2 + 3] = float("nan")                # padding may hold anything
    G.say(f"expert layer held={held} N={N} E={E} K={K} H={H} M={M}")
    out = layer.forward(h, valid=valid)
    dx, dw, _ = layer.backward(dout)
    torch.cuda.synchronize()
    start, src = layer.off.cpu().numpy(), layer.row_src.long()
    assert int(start[-1]) == (N - 3) * K and (src[:int(start[-1])] >= 0).all()
    x = torch.where((src >= 0).unsqueeze(1), h[src.clamp(min=0)].double(), 0.0)
    if held == "bf16":
        xw, wf = x, w.to(torch.bfloat16).double()
        db, wb = layer.drows.double(), wf
    else:
        xw, wf = on_gpu(values(layer.xq, layer.xs))[:, :H], on_gpu(values(layer.wq, layer.ws))[..., :H]
        db = on_gpu(values(layer.dq, layer.ds))[:, :M]
        wb = on_gpu(values(layer.wt, layer.wts))[..., :M].transpose(1, 2).contiguous()
    for e in range(E):
        i, j = int(start[e]), int(start[e + 1])
        if i == j:
            assert (dw[e] == 0).all()
            continue
        close("rows", layer.rows[i:j], xw[i:j] @ wf[e].T, xw[i:j].abs() @ wf[e].abs().T, H)
        close("dx rows", layer.dx_rows[i:j], db[i:j] @ wb[e], db[i:j].abs() @ wb[e].abs(), M)
        d = layer.drows[i:j].double()
        close("dw", dw[e], d.T @ x[i:j], d.abs().T @ x[i:j].abs(), j - i, half=0.0)
    at, live = layer.pos.long().clamp(min=0), (layer.pos >= 0).unsqueeze(2)
    terms = torch.where(live, layer.rows[at].double() * layer.gate.double().unsqueeze(2), 0.0)
    close("out", out, terms.sum(1), terms.abs().sum(1), K)
    back = torch.where(live, layer.dx_rows[at].double(), 0.0)
    close("dx", dx, back.sum(1), back.abs().sum(1), K)
    assert (out[N // 2:N // 2 + 3] == 0).all() and (dx[N // 2:N // 2 + 3] == 0).all()


@pytest.mark.parametrize("held", ["e4m3", "bf16", "e2m1"])
def test_an_update_of_the_matrices(held):
    """Forward, backward, the orthogonalised gradient, the matrices laid out
    again and the bias update, as a training loop runs them, on its own stream."""
    N, E, K, H, M = 500, 32, 4, 256, 96
    layer, w, h, dout = make(N, E, K, H, M, held, 3)
    with pytest.raises(RuntimeError, match="no backward"):
        layer.orthogonalized()
    G.say(f"update of the matrices held={held}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer.forward(h, stream=side)
    _, dw, _ = layer.backward(dout, stream=side)
    o = layer.orthogonalized(stream=side)
    side.synchronize()
    for e in (0, 7, E - 1):
        near_ortho(o[e], dw[e])
    momentum = dw * 0.5
    again = layer.orthogonalized(momentum, stream=side)
    side.synchronize()
    assert again is o
    near_ortho(o[1], momentum[1])
    w.add_(o, alpha=-0.02)
    side.wait_stream(torch.cuda.current_stream())
    layer.load_weights(w, stream=side)
    layer.forward(h, stream=side)
    layer.update_bias(stream=side)
    side.synchronize()
    first = layer.out.clone()
    fresh = ExpertLayer(layer.wr, w, K, N, coef=1e-2, held=held)
    fresh.b.copy_(make(N, E, K, H, M, held, 3)[0].b)
    assert torch.equal(fresh.forward(h), first)
    with pytest.raises(ValueError, match="update has shape"):
        layer.orthogonalized(momentum[:3])


@pytest.mark.parametrize("held", ["bf16", "e2m1"])
def test_the_step_in_a_graph(held):
    N, E, K, H, M = 200, 32, 4, 128, 72
    layer, _, h, dout = make(N, E, K, H, M, held, 5)
    rng = np.random.default_rng(5)
    G.say(f"layer in a graph held={held}")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer.forward(h)
        layer.backward(dout)
        layer.orthogonalized()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.forward(h)
        layer.backward(dout)
        layer.orthogonalized()
    for k in range(4):
        h.copy_(torch.from_numpy(rng.standard_normal((N, H)).astype(np.float32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (layer.out, layer.dx, layer.dw, layer.o)]
        for t in (layer.out, layer.dx, layer.dw, layer.o):
            t.zero_()
        layer.forward(h)
        layer.backward(dout)
        layer.orthogonalized()
        torch.cuda.synchronize()
        for a, b in zip(got, (layer.out, layer.dx, layer.dw, layer.o)):
            assert torch.equal(a, b)
