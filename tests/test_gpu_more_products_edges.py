"""The bf16 and 4-bit products and the orthogonalised update where a caller may
go: numbered rows of an array without any, rows of a few values, arrays beyond
4 GiB, calls on two streams at once and graphs that share a workspace.

Tolerances are those of the products (a sum of n terms in 32 bits is off by
n 2^-23 of their magnitudes, a bf16 result by 2^-8 of it); results of the same
call are compared for equality.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from test_gpu_bf16 import BF16, HALF, data, near, offsets, rows, shifted, taken

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def new(shape, dtype=BF16, value=7):
    return torch.full(shape, value, dtype=dtype, device=G.DEV)


@pytest.mark.parametrize("M,N,C", [(3, 40, 64), (100, 72, 128), (700, 130, 65), (2, 5, 3)])
def test_no_row_to_take(M, N, C):
    """x has no row: every row_src is outside, y is zeros and so is the gradient."""
    rng = np.random.default_rng(1)
    G.say(f"no row to take M={M} N={N} C={C}")
    x, w, dy = torch.empty((0, C), dtype=BF16, device=G.DEV), data(rng, 1, N, C), data(rng, M, N)
    src = G.dev(rng.integers(-1, 4, M).astype(np.int32))
    off = G.dev(np.array([0, M], np.int32))
    for kw, v in ((dict(), w[0]), (dict(off=off), w)):
        y, y_t = new((M, N)), new((M, N))
        qb.qb_bf16_product(x, v, y, row_src=src, **kw)
        qb.qb_bf16_product(x, v.transpose(-1, -2).contiguous(), y_t, row_src=src, transposed=True, **kw)
        dw = new(v.shape, torch.float32)
        qb.qb_bf16_weight_grad(dy, x, dw, row_src=src, **kw)
        torch.cuda.synchronize()
        assert (y == 0).all() and (y_t == 0).all() and (dw == 0).all()
    q, s = new((M, qb.fp4_ld(C)), torch.uint8), new((M, qb.fp4_sld(C)), torch.uint8)
    qb.qb_fp4_quantize(x, q, s, row_src=src)
    torch.cuda.synchronize()
    assert (q[:, :(C + 1) // 2] & 0x77 == 0).all() and (s != 255).all()


@pytest.mark.parametrize("M", [0, 3, 50, 400])
@pytest.mark.parametrize("N,C", [(1, 1), (3, 5), (5, 300), (300, 5), (7, 9), (9, 7), (2, 8), (8, 2), (15, 15)])
def test_rows_of_a_few_values(M, N, C):
    rng = np.random.default_rng(100 * N + C + M)
    E = 3
    off = offsets(rng, E, M, "any") if M else np.zeros(E + 1, np.int32)
    R = int(off[-1])
    G.say(f"rows of a few values M={R} N={N} C={C}")
    x, w, dy, src = data(rng, 20, C), data(rng, E, N, C), data(rng, R, N), rows(rng, R, 20)
    y, dx = new((R, N)), new((R, C))
    dw = new((E, N, C), torch.float32)
    qb.qb_bf16_product(x, w, y, off=G.dev(off), row_src=src)
    qb.qb_bf16_product(dy, w, dx, off=G.dev(off), transposed=True)
    qb.qb_bf16_weight_grad(dy, x, dw, off=G.dev(off), row_src=src)
    torch.cuda.synchronize()
    t = taken(x, src)
    there = ((src >= 0) & (src < 20)).unsqueeze(1)
    for e in range(E):
        i, j = int(off[e]), int(off[e + 1])
        near(y[i:j], t[i:j], w[e].T, HALF)
        near(dx[i:j], dy[i:j], w[e], HALF)
        near(dw[e], (dy * there)[i:j].T, t[i:j], 0.0)


@pytest.mark.parametrize("C", [1024, 1025])
def test_beyond_4_gib(C):
    """Rows whose bytes lie past 2^32, by number and in order."""
    rng = np.random.default_rng(C)
    Mx, N = 2_200_000, 24
    G.say(f"beyond 4 GiB C={C}")
    x = torch.zeros((Mx, C), dtype=BF16, device=G.DEV)
    for a in (0, 1_000_000, 2_097_000, Mx - 500):
        x[a:a + 500] = data(rng, 500, C)
    w = data(rng, N, C)
    for M in (9, 300):
        pick = np.concatenate([rng.integers(0, 500, M // 3), rng.integers(2_097_000, 2_097_500, M // 3),
                               rng.integers(Mx - 500, Mx, M // 3)]).astype(np.int32)
        src, dy = G.dev(pick), data(rng, M, N)
        y, dw = new((M, N)), new((N, C), torch.float32)
        qb.qb_bf16_product(x, w, y, row_src=src)
        qb.qb_bf16_weight_grad(dy, x, dw, row_src=src)
        q, s = new((M, qb.fp4_ld(C)), torch.uint8), new((M, qb.fp4_sld(C)), torch.uint8)
        qb.qb_fp4_quantize(x, q, s, row_src=src)
        t = x[src.long()].contiguous()
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        qb.qb_fp4_quantize(t, q2, s2)
        torch.cuda.synchronize()
        near(y, t, w.T, HALF)
        near(dw, dy.T, t, 0.0)
        assert torch.equal(q, q2) and torch.equal(s, s2)
    y = new((Mx, N))
    qb.qb_bf16_product(x, w, y)
    torch.cuda.synchronize()
    for a in (0, 1_000_000, 2_097_000, Mx - 500):
        near(y[a:a + 500], x[a:a + 500], w.T, HALF)
    assert (y[500:1_000_000] == 0).all()
    del y
    dx = new((Mx, C))                                   # results past 2^32 bytes
    dy = data(rng, Mx, N)
    qb.qb_bf16_product(dy, w, dx, transposed=True)
    torch.cuda.synchronize()
    for a in (0, 2_097_000, Mx - 500):
        near(dx[a:a + 500], dy[a:a + 500], w, HALF)


@pytest.mark.parametrize("M,C", [(5, 33), (130, 256), (700, 1001)])
def test_quantising_at_any_address(M, C):
    rng = np.random.default_rng(M)
    G.say(f"4 bits at any address M={M} C={C}")
    x, w = data(rng, M, C), data(rng, 2, 70, C).float()
    got = []
    for a, b in ((x, w), (shifted(x), shifted(w))):
        q, s = new((M, qb.fp4_ld(C)), torch.uint8), new((M, qb.fp4_sld(C)), torch.uint8)
        wq, ws = new((2, 70, qb.fp4_ld(C)), torch.uint8), new((2, 70, qb.fp4_sld(C)), torch.uint8)
        wt, wts = new((2, C, qb.fp4_ld(70)), torch.uint8), new((2, C, qb.fp4_sld(70)), torch.uint8)
        qb.qb_fp4_quantize(a, q, s)
        qb.qb_fp4_quantize_weight(b, wq, ws, wt, wts)
        y = new((M, 70)) if M != 130 else shifted(new((M, 70)))
        qb.qb_fp4_product(q, s, wq[0].contiguous(), ws[0].contiguous(), y)
        got.append((q, s, wq, ws, wt, wts, y))
    torch.cuda.synchronize()
    for i in range(7):
        assert torch.equal(got[0][i], got[1][i])


class Step:
    """A step of each operator on inputs of its own; the workspace may be another's."""

    def __init__(self, seed, ws=None):
        rng = np.random.default_rng(seed)
        E, N, C, M = 4, 136, 264, 4000
        off = offsets(rng, E, M, "any")
        R = int(off[-1])
        self.off, self.src = G.dev(off), rows(rng, R, 1000)
        self.x, self.w, self.dy = data(rng, 1000, C), data(rng, E, N, C), data(rng, R, N)
        self.f = self.w.float()
        u8 = torch.uint8
        self.q, self.s = new((R, qb.fp4_ld(C)), u8), new((R, qb.fp4_sld(C)), u8)
        self.wq, self.wsc = new((E, N, qb.fp4_ld(C)), u8), new((E, N, qb.fp4_sld(C)), u8)
        self.out = [new((R, N)), new((R, C)), new((E, N, C), torch.float32), new((R, N)), new((E, N, C))]
        need = max(qb.qb_bf16_weight_grad_workspace_bytes(R, N, C, E), qb.qb_orthogonalize_workspace_bytes(E, N, C))
        self.ws = torch.empty((need,), dtype=u8, device=G.DEV) if ws is None else ws
        assert self.ws.numel() >= need

    def run(self, stream=None):
        y, dx, dw, y4, o = self.out
        qb.qb_bf16_product(self.x, self.w, y, off=self.off, row_src=self.src, stream=stream)
        qb.qb_bf16_product(self.dy, self.w, dx, off=self.off, transposed=True, stream=stream)
        qb.qb_bf16_weight_grad(self.dy, self.x, dw, off=self.off, row_src=self.src, ws=self.ws, stream=stream)
        qb.qb_fp4_quantize_weight(self.f, self.wq, self.wsc, stream=stream)
        qb.qb_fp4_quantize(self.x, self.q, self.s, row_src=self.src, stream=stream)
        qb.qb_fp4_product(self.q, self.s, self.wq, self.wsc, y4, off=self.off, stream=stream)
        qb.qb_orthogonalize(self.f, o, self.ws, stream=stream)

    def clear(self):
        for t in self.out:
            t.zero_()

    def kept(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.out]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_streams_at_once():
    G.say("two streams at once")
    steps = [Step(1), Step(2)]
    for s in steps:
        s.run()
    alone = [s.kept() for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in steps:
        s.clear()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, at in zip(steps, streams):
            s.run(at)
    for s, want in zip(steps, alone):
        assert same(s.kept(), want)


def test_graphs_that_share_a_workspace():
    """Two graphs with one workspace, replayed one after the other beside eager work."""
    G.say("graphs that share a workspace")
    first = Step(3)
    steps = [first, Step(4, ws=first.ws)]
    side, graphs = torch.cuda.Stream(), []
    for s in steps:
        s.run()
    alone = [s.kept() for s in steps]
    for s in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s.run()
        graphs.append(graph)
    for _ in range(3):
        for s in steps:
            s.clear()
        first.ws.fill_(0x7F)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        for s, want in zip(steps, alone):
            assert same(s.kept(), want)
