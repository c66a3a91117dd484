"""The expert layer (ExpertLayer): each stage of a training step against its
definition in float64, from the values that the stage before left, the bias
update against the oracle, and the whole step in a captured graph.

Tolerances: a bf16 result is off by half a step, 2^-8 of it; a sum of n terms
in 32 bits by n 2^-23 of their magnitudes; the 8-bit instruction may drop
8 2^-13 = 2^-10 of them more (see the products' own tests).
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb
from exact_quantile_selection_amd.expert_layer import ExpertLayer

import gpu_util as G

pytestmark = pytest.mark.gpu
STEP, HALF, DROP = 2.0 ** -23, 2.0 ** -8, 2.0 ** -10


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def close(name, got, ref, mag, n, half=HALF, drop=0.0):
    off = (got.double() - ref).abs() - (half * ref.abs() + (n * STEP + drop) * mag)
    assert not torch.isnan(got).any(), name
    assert (off <= 0).all(), f"{name}: {(off > 0).sum().item()} of {off.numel()} off"


def held(q, s, rows_a_scale=1):
    """What e4m3 q [.., rows, ld] with its scale bytes stands for, float64."""
    e = s.double()[..., :q.shape[-1] // 128] - 127
    e = e.repeat_interleave(rows_a_scale, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)
    return q.float().double() * torch.exp2(e)


def make(N, E, K, H, M, B, seed):
    g = torch.Generator(device=G.DEV).manual_seed(seed)
    wr = torch.randn((E, H), generator=g, device=G.DEV) / H ** 0.5
    w = torch.randn((E, M, H), generator=g, device=G.DEV) / H ** 0.5
    layer = ExpertLayer(wr.to(torch.bfloat16), w, K, N, coef=1e-2, B=B)
    layer.b.copy_((torch.rand(E, generator=g, device=G.DEV) - 0.5) * 0.1)
    h = torch.randn((N, H), generator=g, device=G.DEV).to(torch.bfloat16)
    dout = torch.randn((N, M), generator=g, device=G.DEV).to(torch.bfloat16)
    return layer, h, dout


@pytest.mark.parametrize("N,E,K,H,M", [(300, 32, 2, 256, 200), (1000, 64, 6, 512, 130), (16, 256, 8, 256, 384)])
def test_a_training_step(O, N, E, K, H, M):
    B = 3
    layer, h, dout = make(N, E, K, H, M, B, N + E)
    off = torch.tensor([0, N // 4, N // 4, N], dtype=torch.int32, device=G.DEV)
    valid = torch.ones(N, dtype=torch.uint8, device=G.DEV)
    valid[N // 2:N // 2 + 3] = 0
    dloss = torch.full((1,), 64.0, device=G.DEV)
    G.say(f"expert layer N={N} E={E} K={K} H={H} M={M}")
    out = layer.forward(h, seq_off=off, valid=valid)
    dx, dw, dlogits = layer.backward(dout, dloss)
    torch.cuda.synchronize()

    # the order: every live pair has a row of its expert, every other row none
    topk, pos = layer.topk.cpu().numpy(), layer.pos.cpu().numpy()
    start, src = layer.off.cpu().numpy(), layer.row_src.cpu().numpy()
    live = valid.cpu().numpy() != 0
    assert ((topk >= 0) == live[:, None]).all() and ((pos >= 0) == live[:, None]).all()
    t = np.repeat(np.arange(N), K).reshape(N, K)
    assert (src[pos[live]] == t[live]).all() and (src >= 0).sum() == live.sum() * K
    assert ((start[topk[live]] <= pos[live]) & (pos[live] < start[topk[live] + 1])).all()
    assert layer.count.sum().item() == live.sum() * K

    # the experts' rows and their sum
    x = held(layer.xq, layer.xs)
    w, wt = held(layer.wq, layer.ws, 128), held(layer.wt, layer.wts, 128)
    d, xt, dt = held(layer.dq, layer.ds), held(layer.xt, layer.xts), held(layer.dt, layer.dts)
    for e in range(E):
        i, j = int(start[e]), int(start[e + 1])
        close("rows", layer.rows[i:j], x[i:j] @ w[e].T, x[i:j].abs() @ w[e].abs().T, H, drop=DROP)
        close("dx rows", layer.dx_rows[i:j], d[i:j] @ wt[e].T, d[i:j].abs() @ wt[e].abs().T, M, drop=DROP)
        a, b = dt[:, i:j], xt[:, i:j]
        close("dw", dw[e], a @ b.T, a.abs() @ b.abs().T, j - i, half=0.0)
    at, on = layer.pos.long().clamp(min=0), (layer.pos >= 0).unsqueeze(2)
    zero = torch.zeros((), dtype=torch.float64, device=G.DEV)
    picked = torch.where(on, layer.rows[at].double(), zero)
    terms = picked * layer.gate.double().unsqueeze(2)
    close("out", out, terms.sum(1), terms.abs().sum(1), K)
    back = torch.where(on, layer.dx_rows[at].double(), zero)
    close("dx", dx, back.sum(1), back.abs().sum(1), K)

    # the gates' gradient and the router's, by the formulas of the balance loss
    prod = picked * dout.double().unsqueeze(1)
    close("dgate", layer.dgate, prod.sum(2), prod.abs().sum(2), M, half=0.0)
    lv = valid.bool().unsqueeze(1)
    seq = (torch.arange(N, device=G.DEV) >= N // 4).long() * 2
    s, weight = layer.s.double(), (layer.weight.double() * dloss.double())[seq]
    z = s.sum(1, keepdim=True)
    chosen = layer.topk.long().clamp(min=0)
    mine = torch.gather(s, 1, chosen)
    gate, dg = mine / mine.sum(1, keepdim=True), layer.dgate.double()
    ds = (weight - (weight * s / z).sum(1, keepdim=True)) / z
    add = (dg - (dg * gate).sum(1, keepdim=True)) / mine.sum(1, keepdim=True)
    size = (weight.abs() + (weight.abs() * s / z).sum(1, keepdim=True)) / z
    size = size.scatter_add(1, chosen, (dg.abs() + (dg.abs() * gate).sum(1, keepdim=True)) / mine.sum(1, keepdim=True))
    ref = torch.where(lv, ds.scatter_add(1, chosen, add) * s * (1 - s), zero)
    close("dlogits", dlogits, ref, torch.where(lv, size * s * (1 - s), zero), 20, half=0.0)

    # the bias update of the same scores
    want = O.eqb_layer(layer.s.cpu().numpy(), layer.b.cpu().numpy(), K)
    layer.update_bias()
    torch.cuda.synchronize()
    G.assert_same("b", layer.b.cpu().numpy(), want["b_next"])


def test_the_step_in_a_graph():
    """Three replays, other inputs copied in each time and eager steps of a
    second layer between them, each equal to the eager step on a side stream."""
    N, E, K, H, M = 200, 32, 4, 256, 130
    layer, h, dout = make(N, E, K, H, M, 1, 7)
    other, h2, dout2 = make(N, E, K, H, M, 1, 8)
    names = ("out", "loss", "dx", "dw", "dlogits", "b")

    def step(l, x, d):
        l.forward(x)
        l.backward(d)
        l.update_bias()

    b0 = layer.b.clone()
    G.say("expert layer in a graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer, h, dout)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layer, h, dout)
    for k in range(3):
        g = torch.Generator(device=G.DEV).manual_seed(100 + k)
        h.copy_(torch.randn((N, H), generator=g, device=G.DEV))
        dout.copy_(torch.randn((N, M), generator=g, device=G.DEV))
        layer.b.copy_(b0)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: getattr(layer, n).clone() for n in names}
        step(other, h2, dout2)
        layer.b.copy_(b0)
        for n in names[:-1]:
            getattr(layer, n).fill_(float("nan"))
        with torch.cuda.stream(side):
            step(layer, h, dout)
        torch.cuda.synchronize()
        for n in names:
            G.assert_same(n, got[n].float().cpu().numpy(), getattr(layer, n).float().cpu().numpy())
