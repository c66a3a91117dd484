"""The experts' products in bfloat16 (qb_bf16_*) against their definition in
float64.

A product of two bf16 values is exact in 32 bits; a sum of n of them adds n
terms, each addition off by at most one step, 2^-23 of the terms' magnitudes:
n 2^-23 sum |a b| in 32 bits, and half a bf16 step, 2^-8 of the result, where
it is rounded to bf16.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu
STEP, HALF = 2.0 ** -23, 2.0 ** -8
BF16, NAN = torch.bfloat16, float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(G.DEV)


def data(rng, *shape):
    """Rows and columns of different sizes, some zeros."""
    x = randn(rng, *shape) * torch.exp(randn(rng, *shape[:-1], 1)) * torch.exp(randn(rng, shape[-1]))
    x[randn(rng, *shape) > 1.6] = 0
    return x.to(BF16)


def shifted(t):
    """The same values one element off a 16-byte boundary."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = flat[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    return out


def near(got, a, b, half):
    """got [i, j] against sum_k a[i, k] b[k, j]."""
    a, b = a.double(), b.double()
    ref, mag = a @ b, a.abs() @ b.abs()
    off = (got.double() - ref).abs() - (half * ref.abs() + a.shape[1] * STEP * mag)
    assert not torch.isnan(got).any() and (off.numel() == 0 or off.max().item() <= 0), (
        f"{(off > 0).sum().item()} of {off.numel()} off")


def rows(rng, M, Mx, bad=True):
    """Row numbers in any order, some outside."""
    src = rng.integers(-2 if bad else 0, Mx + (2 if bad else 0), M).astype(np.int32)
    return G.dev(src)


def taken(x, src):
    """x's rows by number, zeros outside."""
    if src is None:
        return x
    src = src.long()
    inside = ((src >= 0) & (src < x.shape[0])).unsqueeze(1)
    return torch.where(inside, x[src.clamp(0, x.shape[0] - 1)], torch.zeros((), dtype=x.dtype, device=x.device))


def offsets(rng, E, M, kind, align=1):
    if kind == "one":                                  # everything at the last expert
        c = np.zeros(E, np.int64)
        c[-1] = M
    else:
        w = np.exp(1.5 * rng.standard_normal(E)) * (rng.random(E) > 0.4)
        w[rng.integers(E)] += 1
        c = rng.multinomial(M, w / w.sum())
    c = -(-c // align) * align
    return np.concatenate([[0], np.cumsum(c)]).astype(np.int32)


# sizes on both sides of each kind of kernel, odd ones, single rows and columns
SIZES = [(1, 1, 1), (1, 16, 128), (1, 4096, 1024), (5, 33, 300), (16, 17, 2000), (17, 256, 640), (33, 130, 129),
         (64, 200, 512), (65, 136, 704), (200, 704, 136), (777, 2005, 1001), (129, 1, 4096), (1000, 2056, 264),
         (3000, 4100, 260), (4000, 4096, 512)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,N,C", SIZES)
def test_product(M, N, C, transposed):
    rng = np.random.default_rng(M + N + C)
    G.say(f"bf16 product M={M} N={N} C={C} transposed={transposed}")
    w = data(rng, N, C) if not transposed else data(rng, C, N)
    for src in (None, rows(rng, M, M // 2 + 1)):
        x = data(rng, M if src is None else M // 2 + 1, C)
        y = torch.full((M, N), NAN, dtype=BF16, device=G.DEV)
        qb.qb_bf16_product(x, w, y, row_src=src, transposed=transposed)
        torch.cuda.synchronize()
        near(y, taken(x, src), w if transposed else w.T, HALF)


EXPERTS = [(1, 3, 16, 128), (256, 128, 64, 520), (16, 300, 130, 200), (16, 700, 104, 304), (7, 2000, 260, 257),
           (32, 9000, 520, 384), (256, 5000, 33, 130), (3, 6000, 1024, 520)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("kind", ["any", "one"])
@pytest.mark.parametrize("E,M,N,C", EXPERTS)
def test_product_of_experts(E, M, N, C, kind, transposed):
    rng = np.random.default_rng(E + M)
    off = offsets(rng, E, M, kind)
    R = int(off[-1]) + 5                               # rows past the last expert stay as they were
    G.say(f"bf16 experts' product E={E} M={R} N={N} C={C} {kind} transposed={transposed}")
    w = data(rng, E, N, C) if not transposed else data(rng, E, C, N)
    for src in (None, rows(rng, R, 50)):
        x = data(rng, R if src is None else 50, C)
        if src is None:
            x[off[-1]:] = NAN                          # and are not multiplied
        y = torch.full((R, N), 77.0, dtype=BF16, device=G.DEV)
        qb.qb_bf16_product(x, w, y, off=G.dev(off), row_src=src, transposed=transposed)
        torch.cuda.synchronize()
        t = taken(x, src)
        for e in range(E):
            i, j = int(off[e]), int(off[e + 1])
            if i < j:
                near(y[i:j], t[i:j], w[e] if transposed else w[e].T, HALF)
        assert (y[off[-1]:] == 77.0).all()


@pytest.mark.parametrize("M,N,C", [(5, 33, 304), (70, 128, 64), (300, 264, 512)])
def test_arrays_at_any_address(M, N, C):
    rng = np.random.default_rng(M)
    G.say(f"bf16 unaligned M={M} N={N} C={C}")
    x, w, dy = data(rng, M, C), data(rng, N, C), data(rng, M, N)
    y, dx = shifted(torch.zeros_like(dy)), shifted(torch.zeros_like(x))
    dw = shifted(torch.zeros((N, C), dtype=torch.float32, device=G.DEV))
    qb.qb_bf16_product(shifted(x), shifted(w), y)
    qb.qb_bf16_product(shifted(dy), shifted(w), dx, transposed=True)
    qb.qb_bf16_weight_grad(shifted(dy), shifted(x), dw)
    torch.cuda.synchronize()
    near(y, x, w.T, HALF)
    near(dx, dy, w, HALF)
    near(dw, dy.T, x, 0.0)


@pytest.mark.parametrize("M,N,C", [(1, 1, 1), (5, 16, 700), (128, 130, 65), (777, 505, 301), (640, 2104, 1032),
                                   (2000, 3, 4097), (3001, 72, 136), (20000, 128, 64), (4000, 2048, 2056), (300, 4104, 4096)])
def test_weight_gradient(M, N, C):
    rng = np.random.default_rng(M + N + C)
    G.say(f"bf16 weight gradient M={M} N={N} C={C}")
    dy = data(rng, M, N)
    ws = torch.empty(qb.qb_bf16_weight_grad_workspace_bytes(M, N, C), dtype=torch.uint8, device=G.DEV)
    for src in (None, rows(rng, M, M // 2 + 1)):
        x = data(rng, M if src is None else M // 2 + 1, C)
        d = dy.clone()
        if src is not None:
            out = (src < 0) | (src >= x.shape[0])
            d[out] = NAN                               # a row that was routed nowhere adds nothing
        for w in (None, ws):
            dw = torch.full((N, C), NAN, dtype=torch.float32, device=G.DEV)
            qb.qb_bf16_weight_grad(d, x, dw, row_src=src, ws=w)
            torch.cuda.synchronize()
            near(dw, torch.where(torch.isnan(d), 0.0, d.double()).T, taken(x, src), 0.0)


@pytest.mark.parametrize("kind", ["any", "one"])
@pytest.mark.parametrize("E,M,N,C", EXPERTS + [(2, 9000, 64, 72), (5, 4000, 33, 47)])
def test_weight_gradient_of_experts(E, M, N, C, kind):
    rng = np.random.default_rng(E + M)
    off = offsets(rng, E, M, kind)
    R = int(off[-1]) + 5
    G.say(f"bf16 experts' weight gradient E={E} M={R} N={N} C={C} {kind}")
    ws = torch.empty(qb.qb_bf16_weight_grad_workspace_bytes(R, N, C, E), dtype=torch.uint8, device=G.DEV)
    for src, w in ((None, None), (rows(rng, R, 50), None), (rows(rng, R, 50), ws)):
        x, dy = data(rng, R if src is None else 50, C), data(rng, R, N)
        dy[off[-1]:] = NAN
        dw = torch.full((E, N, C), NAN, dtype=torch.float32, device=G.DEV)
        qb.qb_bf16_weight_grad(dy, x, dw, off=G.dev(off), row_src=src, ws=w)
        torch.cuda.synchronize()
        t = taken(x, src)
        for e in range(E):
            i, j = int(off[e]), int(off[e + 1])
            if i < j:
                near(dw[e], dy[i:j].T, t[i:j], 0.0)
            else:
                assert (dw[e] == 0).all()


def test_neighbours_and_infinities_stay_where_they_are():
    """Infinities and NaN of one expert's rows, and of one row, reach no other."""
    rng = np.random.default_rng(5)
    E, N, C = 4, 136, 72
    off = np.array([0, 70, 70, 201, 333], np.int32)
    x, w, dy = data(rng, 333, C), data(rng, E, N, C), data(rng, 333, N)
    x[70:201:3], dy[70:201:5], w[1] = NAN, float("inf"), NAN
    G.say("bf16 infinities")
    y, dw = torch.zeros((333, N), dtype=BF16, device=G.DEV), torch.zeros((E, N, C), device=G.DEV)
    dx = torch.zeros((333, C), dtype=BF16, device=G.DEV)
    qb.qb_bf16_product(x, w, y, off=G.dev(off))
    qb.qb_bf16_product(dy, w, dx, off=G.dev(off), transposed=True)
    qb.qb_bf16_weight_grad(dy, x, dw, off=G.dev(off))
    torch.cuda.synchronize()
    for i, j, e in ((0, 70, 0), (201, 333, 3)):
        near(y[i:j], x[i:j], w[e].T, HALF)
        near(dx[i:j], dy[i:j], w[e], HALF)
        near(dw[e], dy[i:j].T, x[i:j], 0.0)
    good = [i for i in range(70, 201) if (i - 70) % 3]
    near(y[good], x[good], w[2].T, HALF)
    assert torch.isnan(y[70:201:3]).all() and not torch.isfinite(dw[2]).any()


def test_gradients_against_differences():
    """d/dx and d/dw of sum(y g), y in float64 by the definition: the loss is
    bilinear, so a difference of any length is its derivative."""
    rng = np.random.default_rng(9)
    E, M, N, C = 3, 90, 24, 40
    off = np.array([0, 33, 34, 90], np.int32)
    src = rows(rng, M, 60, bad=False)
    x, w, dy = data(rng, 60, C), data(rng, E, N, C), data(rng, M, N)
    dx, dw = torch.zeros((M, C), dtype=BF16, device=G.DEV), torch.zeros((E, N, C), device=G.DEV)
    G.say("bf16 differences")
    qb.qb_bf16_product(dy, w, dx, off=G.dev(off), transposed=True)
    qb.qb_bf16_weight_grad(dy, x, dw, off=G.dev(off), row_src=src)
    torch.cuda.synchronize()

    def loss(xr, wd):
        return sum(((xr[i:j] @ wd[e].T) * dy[i:j].double()).sum() for e, (i, j) in enumerate(zip(off, off[1:])))

    xr, wd = taken(x, src).double(), w.double()
    for k in range(20):
        v, u = randn(rng, M, C).double(), randn(rng, E, N, C).double()
        one = (loss(xr + v, wd) - loss(xr - v, wd)) / 2
        mag = sum(((dy[i:j].double().abs() @ wd[e].abs()) * v[i:j].abs()).sum() for e, (i, j) in enumerate(zip(off, off[1:])))
        # half a bf16 step of each value of dx, and the sum's own 32 bits
        assert abs(one - (dx.double() * v).sum()) <= HALF / (1 - HALF) * (dx.double() * v).abs().sum() + N * STEP * mag
        two = (loss(xr, wd + u) - loss(xr, wd - u)) / 2
        mag = sum(((dy[i:j].double().abs().T @ xr[i:j].abs()) * u[e].abs()).sum() for e, (i, j) in enumerate(zip(off, off[1:])))
        assert abs(two - (dw.double() * u).sum()) <= M * STEP * mag


def test_captured_and_on_another_stream():
    """Calls of a graph, replayed beside eager work, on a stream of their own."""
    rng = np.random.default_rng(11)
    E, N, C = 5, 128, 192
    off = offsets(rng, E, 900, "any")
    R = int(off[-1])
    w, offd, src = data(rng, E, N, C), G.dev(off), rows(rng, R, 300)
    x, dy = data(rng, 300, C), data(rng, R, N)
    y, dx = torch.zeros((R, N), dtype=BF16, device=G.DEV), torch.zeros((R, C), dtype=BF16, device=G.DEV)
    dw = torch.zeros((E, N, C), device=G.DEV)
    ws = torch.empty(qb.qb_bf16_weight_grad_workspace_bytes(R, N, C, E), dtype=torch.uint8, device=G.DEV)

    def step(stream=None):
        qb.qb_bf16_product(x, w, y, off=offd, row_src=src, stream=stream)
        qb.qb_bf16_product(dy, w, dx, off=offd, transposed=True, stream=stream)
        qb.qb_bf16_weight_grad(dy, x, dw, off=offd, row_src=src, ws=ws, stream=stream)

    G.say("bf16 graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in range(4):
        x.copy_(data(rng, 300, C))
        dy.copy_(data(rng, R, N))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        for t in (y, dx, dw):
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        side.synchronize()
        for a, b in zip(got, (y, dx, dw)):
            assert torch.equal(a, b)
