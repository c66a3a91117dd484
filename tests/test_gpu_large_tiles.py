"""The products' largest tiles, 256 x 256, where they have something left over:
the matrices' gradient of one matrix and of experts, and rows by number from
arrays of 2 to 4 GiB, whose 32-bit offsets the loads to LDS take.

Tolerances are those of test_gpu_bf16.py.  Which kernel ran is read from a trace
of the call, so that another rule for the tiles cannot leave this one untested.
"""
import re

import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from test_gpu_bf16 import BF16, HALF, NAN, data, near, offsets, rows, taken

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def tile(call):
    """The edge of the tiles that `call` ran, None where this machine gives no trace."""
    from torch.profiler import ProfilerActivity, profile

    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    names = [e.name for e in p.events() if "k_gemm16" in e.name]
    # (a name is written out or not: k_gemm16<.., true, true, 256, ..>, k_gemm16I..Lb1ELb1ELi256E..)
    return int(re.search(r"(?<!\d)(64|128|256)(?!\d)", names[0]).group(1)) if names else None


def ran(call, B):
    assert tile(call) in (B, None)


def numbered(rng, R, Mx, dy):
    """Row numbers, some outside, whose rows of dy hold NaN."""
    src = rows(rng, R, Mx)
    src[1::17], src[2::29] = -1, Mx
    dy = dy.clone()
    dy[(src < 0) | (src >= Mx)] = NAN
    return src, dy


def gradient_of(dy, x, src):
    return torch.where(torch.isnan(dy), torch.zeros((), dtype=BF16, device=dy.device), dy), taken(x, src)


@pytest.mark.parametrize("M,N,C", [(333, 4088, 4096), (5, 4096, 4088), (64, 4096, 4096), (1500, 3848, 4096)])
def test_gradient_of_one_matrix(M, N, C):
    rng = np.random.default_rng(M)
    G.say(f"bf16 weight gradient in tiles of 256, M={M} N={N} C={C}")
    dy, dw = data(rng, M, N), torch.full((N, C), NAN, dtype=torch.float32, device=G.DEV)
    for src, d, x in ((None, dy, data(rng, M, C)), numbered(rng, M, 50, dy) + (data(rng, 50, C),)):
        dw.fill_(NAN)
        ran(lambda: qb.qb_bf16_weight_grad(d, x, dw, row_src=src), 256)
        a, b = gradient_of(d, x, src)
        near(dw, a.T, b, 0.0)


@pytest.mark.parametrize("kind", ["any", "one", "short"])
@pytest.mark.parametrize("E,M,N,C", [(16, 3000, 2040, 1016), (16, 700, 2048, 1024)])
def test_gradient_of_experts(E, M, N, C, kind):
    rng = np.random.default_rng(M)
    if kind == "short":                                # single rows, whole stages, and nothing
        c = rng.permutation(np.array([0, 1, 63, 64, 65, 0, 128, 2] * (E // 8)))
        off = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    else:
        off = offsets(rng, E, M, kind)
    R = int(off[-1]) + 7
    G.say(f"bf16 experts' weight gradient in tiles of 256, E={E} M={R} N={N} C={C} {kind}")
    dy, dw = data(rng, R, N), torch.full((E, N, C), NAN, dtype=torch.float32, device=G.DEV)
    for src, d, x in ((None, dy, data(rng, R, C)), numbered(rng, R, 50, dy) + (data(rng, 50, C),)):
        d[off[-1]:] = NAN                              # rows behind the last expert
        dw.fill_(NAN)
        ran(lambda: qb.qb_bf16_weight_grad(d, x, dw, off=G.dev(off), row_src=src), 256)
        a, b = gradient_of(d, x, src)
        for e in range(E):
            i, j = int(off[e]), int(off[e + 1])
            if i < j:
                near(dw[e], a[i:j].T, b[i:j], 0.0)
            else:
                assert (dw[e] == 0).all()


def test_not_finite_values_stay_with_their_expert():
    rng = np.random.default_rng(3)
    E, N, C = 16, 2040, 1016
    off = np.arange(E + 1, dtype=np.int32) * 100
    G.say("bf16 weight gradient in tiles of 256, infinities")
    x, dy, dw = data(rng, 100 * E, C), data(rng, 100 * E, N), torch.zeros((E, N, C), device=G.DEV)
    x[300:400:3], dy[500:600:7] = NAN, float("inf")
    ran(lambda: qb.qb_bf16_weight_grad(dy, x, dw, off=G.dev(off)), 256)
    for e in range(E):
        if e == 3:
            assert torch.isnan(dw[e]).all()
        elif e == 5:
            assert not torch.isfinite(dw[e]).all()
        else:
            near(dw[e], dy[100 * e:100 * e + 100].T, x[100 * e:100 * e + 100], 0.0)


def test_the_gradient_in_a_graph():
    """Replayed beside eager work, with other inputs each time."""
    rng = np.random.default_rng(4)
    E, N, C = 16, 2040, 1016
    off = offsets(rng, E, 900, "any")
    R = int(off[-1])
    offd, (src, _) = G.dev(off), numbered(rng, R, 300, torch.zeros((R, 1), device=G.DEV))
    x, dy, dw = data(rng, 300, C), data(rng, R, N), torch.zeros((E, N, C), device=G.DEV)
    G.say("bf16 weight gradient in tiles of 256, graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        qb.qb_bf16_weight_grad(dy, x, dw, off=offd, row_src=src)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qb.qb_bf16_weight_grad(dy, x, dw, off=offd, row_src=src)
    for _ in range(3):
        x.copy_(data(rng, 300, C))
        dy.copy_(data(rng, R, N))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = dw.clone()
        dw.zero_()
        qb.qb_bf16_weight_grad(dy, x, dw, off=offd, row_src=src)
        torch.cuda.synchronize()
        assert torch.equal(got, dw)


def test_rows_by_number_up_to_4_gib():
    """An array of 2^32 bytes: the last whose rows' offsets fit the loads to LDS."""
    rng = np.random.default_rng(7)
    Mx, C = 1 << 22, 512
    G.say("rows by number up to 4 GiB")
    x = torch.zeros((Mx, C), dtype=BF16, device=G.DEV)
    far = (0, (1 << 21) - 250, 3_000_000, Mx - 500)    # both sides of 2 GiB
    for a in far:
        x[a:a + 500] = data(rng, 500, C)
    for M, N, B in ((3000, 264, 64), (20000, 2048, 256)):
        pick = np.concatenate([rng.integers(a, a + 500, M // 4) for a in far])
        src = G.dev(rng.permutation(pick).astype(np.int32))
        w, dy, y = data(rng, N, C), data(rng, M, N), torch.full((M, N), NAN, dtype=BF16, device=G.DEV)
        ran(lambda: qb.qb_bf16_product(x, w, y, row_src=src), B)
        t = x[src.long()]
        near(y, t, w.T, HALF)
        dw = torch.full((N, C), NAN, dtype=torch.float32, device=G.DEV)
        qb.qb_bf16_weight_grad(dy, x, dw, row_src=src)
        torch.cuda.synchronize()
        near(dw, dy.T, t, 0.0)
    # the experts' gradient in tiles of 256 reads them too
    E, N = 32, 2048
    off = offsets(rng, E, 3000, "any")
    src = G.dev(rng.permutation(np.concatenate([rng.integers(a, a + 500, 750) for a in far])).astype(np.int32))
    dy, dw = data(rng, 3000, N), torch.full((E, N, C), NAN, dtype=torch.float32, device=G.DEV)
    ran(lambda: qb.qb_bf16_weight_grad(dy, x, dw, off=G.dev(off), row_src=src), 256)
    t = x[src.long()]
    for e in range(E):
        i, j = int(off[e]), int(off[e + 1])
        if i < j:
            near(dw[e], dy[i:j].T, t[i:j], 0.0)
        else:
            assert (dw[e] == 0).all()
