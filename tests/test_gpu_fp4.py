"""Products in 4-bit floating point with a power-of-two scale for each block of
32 (qb_fp4_*) against their definition in float64.

A quantised value is exact: the scale is the least power of two that keeps the
block within 6, and the value is rounded to nearest even on e2m1's grid, so both
are compared for equality.  A product of two such values is exact in 32 bits; a
sum of n of them adds n terms, each addition off by at most one step, 2^-23 of
the terms' magnitudes: n 2^-23 sum |a b| in 32 bits, and half a bf16 step, 2^-8
of the result, where it is rounded to bf16.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu
STEP, HALF = 2.0 ** -23, 2.0 ** -8
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def bf16_values(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def exponent(top):
    """The least whole e >= -126 with top <= 6 * 2^e (float64, finite)."""
    e = np.full(top.shape, -126)
    for k in range(-126, 127):
        e = np.where(top > 6.0 * 2.0 ** k, k + 1, e)
    return e


def e2m1(v):
    """Nearest even of the grid, |v| <= 6."""
    a = np.abs(v)
    far = np.abs(a[..., None] - GRID)
    far[..., 1::2] += 1e-300                           # equally near: the even number
    best = far.min(-1, keepdims=True)
    pick = np.where((far[..., 0::2] <= best).any(-1), 2 * (far[..., 0::2] <= best).argmax(-1), far.argmin(-1))
    return np.sign(v) * GRID[pick]


def quantise(x):
    """x [rows, n] float64 -> the values it stands for [rows, 2 ld], exponents [rows, blocks]."""
    rows, n = x.shape
    t = np.zeros((rows, 2 * qb.fp4_ld(n)))
    t[:, :n] = x
    t = t.reshape(rows, -1, 32)
    e = exponent(np.abs(t).max(2))
    return (e2m1(t / 2.0 ** e[..., None]) * 2.0 ** e[..., None]).reshape(rows, -1), e


def values(q, s):
    """What e2m1 q [.., rows, ld] with scale bytes s [.., rows, sld] stands for, float64."""
    q, s = G.host(q), G.host(s).astype(np.float64)
    code = np.stack([q & 15, q >> 4], -1).reshape(q.shape[:-1] + (-1,))
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    scale = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return v * np.repeat(scale, 32, -1)


def new_quantised(rows, n, lead=()):
    q = torch.full(lead + (rows, qb.fp4_ld(n)), 0x55, dtype=torch.uint8, device=G.DEV)
    return q, torch.full(lead + (rows, qb.fp4_sld(n)), 255, dtype=torch.uint8, device=G.DEV)


def data(rng, M, C):
    """Rows and columns of very different sizes, zeros, values at the border
    of a scale and between the grid's."""
    x = rng.standard_normal((M, C)) * np.exp(2 * rng.standard_normal((M, 1))) * np.exp(rng.standard_normal((1, C)))
    x[rng.random((M, C)) < 0.05] = 0
    if M > 3:
        x[1] = 6.0 * 2.0 ** rng.integers(-4, 4, C)
        x[2] = rng.integers(-24, 25, C) * 0.25
        x[3] = 0
    return bf16_values(x)


@pytest.mark.parametrize("M,C", [(1, 1), (1, 4096), (3, 31), (5, 32), (130, 257), (777, 1001), (2100, 520), (9, 5000)])
def test_quantising_is_exact(M, C):
    rng = np.random.default_rng(M + C)
    x = data(rng, M, C)
    G.say(f"quantise M={M} C={C}")
    q, s = new_quantised(M, C)
    qb.qb_fp4_quantize(x.to(G.DEV), q, s)
    torch.cuda.synchronize()
    want, e = quantise(x.double().numpy())
    G.assert_same("exponents", G.host(s).astype(np.int64) - 127, e.astype(np.int64))
    assert np.array_equal(values(q, s), want)


def test_every_pattern():
    """Every finite bf16 value beside block maxima that give each a scale near
    its own size and far from it."""
    p = np.arange(0x8000, dtype=np.uint32)
    p = p[p < 0x7F80]
    x = torch.from_numpy((p << 16).astype(np.uint32).view(np.float32)).double().numpy()
    rows = []
    for f in (0.0, 1.0, 2.0, 5.0, 16.0, 100.0):
        t = np.zeros((len(x), 32))
        t[:, 3], t[:, 4] = x, -x
        t[:, 9] = np.minimum(f * x, float(torch.finfo(torch.bfloat16).max))
        rows.append(bf16_values(t))
    x = torch.cat(rows)
    G.say("quantise every pattern")
    q, s = new_quantised(len(x), 32)
    qb.qb_fp4_quantize(x.to(G.DEV), q, s)
    torch.cuda.synchronize()
    want, e = quantise(x.double().numpy())
    G.assert_same("exponents", G.host(s)[:, 0].astype(np.int64) - 127, e[:, 0].astype(np.int64))
    assert np.array_equal(values(q, s), want)


def test_a_block_that_is_not_finite():
    x = torch.ones((4, 96), dtype=torch.bfloat16)
    x[1, 40], x[2, 0], x[3, 95] = float("nan"), float("inf"), -float("inf")
    w = torch.ones((2, 96))
    w[1, 33] = float("nan")
    G.say("quantise NaN")
    q, s = new_quantised(4, 96)
    wq, ws = new_quantised(2, 96)
    wt, wts = new_quantised(96, 2)
    qb.qb_fp4_quantize(x.to(G.DEV), q, s)
    qb.qb_fp4_quantize_weight(w.to(G.DEV), wq, ws, wt, wts)
    y = torch.zeros((4, 2), dtype=torch.bfloat16, device=G.DEV)
    qb.qb_fp4_product(q, s, wq, ws, y)
    torch.cuda.synchronize()
    nan = torch.zeros((4, 8), dtype=torch.bool)
    nan[1, 1], nan[2, 0], nan[3, 2] = True, True, True
    assert torch.equal(s.cpu() == 255, nan)
    assert (ws.cpu() == 255).sum() == 1 and ws[1, 1] == 255
    assert (wts.cpu() == 255).sum() == 1 and wts[33, 0] == 255
    assert torch.equal(torch.isnan(y).cpu(), torch.tensor([[False, True], [True] * 2, [True] * 2, [True] * 2]))
    assert y[0, 0] == 96


def test_rows_by_number():
    rng = np.random.default_rng(3)
    Mx, M, C = 90, 300, 333
    x = data(rng, Mx, C)
    src = rng.integers(-2, Mx + 2, M).astype(np.int32)
    picked = np.where(((src >= 0) & (src < Mx))[:, None], x.double().numpy()[np.clip(src, 0, Mx - 1)], 0)
    G.say("quantise by row number")
    q, s = new_quantised(M, C)
    qb.qb_fp4_quantize(x.to(G.DEV), q, s, row_src=G.dev(src))
    torch.cuda.synchronize()
    assert np.array_equal(values(q, s), quantise(picked)[0])


@pytest.mark.parametrize("lead,N,C", [((), 1, 1), ((), 130, 700), ((3,), 257, 128), ((2,), 64, 1030), ((1,), 1000, 33)])
def test_weights_in_both_orders(lead, N, C):
    rng = np.random.default_rng(N + C)
    w = (rng.standard_normal(lead + (N, C)) * np.exp(2 * rng.standard_normal(lead + (N, 1)))).astype(np.float32)
    G.say(f"quantise weight {lead} {N} {C}")
    (q, s), (qt, st) = new_quantised(N, C, lead), new_quantised(C, N, lead)
    qb.qb_fp4_quantize_weight(G.dev(w), q, s, qt, st)
    alone, sa = new_quantised(N, C, lead)
    qb.qb_fp4_quantize_weight(G.dev(w), alone, sa)
    torch.cuda.synchronize()
    assert torch.equal(alone, q) and torch.equal(s, sa)
    got, gt, w64 = values(q, s), values(qt, st), w.astype(np.float64)
    for g in np.ndindex(*lead):
        want, e = quantise(w64[g])
        assert np.array_equal(got[g], want) and np.array_equal(G.host(s)[g].astype(np.int64) - 127, e)
        want, e = quantise(w64[g].T)
        assert np.array_equal(gt[g], want) and np.array_equal(G.host(st)[g].astype(np.int64) - 127, e)


def weight(rng, N, C, lead=()):
    """A laid out weight and its float64 values."""
    w = rng.standard_normal(lead + (N, C)) * np.exp(rng.standard_normal(lead + (N, 1))) / np.sqrt(C)
    q, s = new_quantised(N, C, lead)
    qb.qb_fp4_quantize_weight(G.dev(w.astype(np.float32)), q, s)
    torch.cuda.synchronize()
    return q, s, values(q, s)


def quantised(x):
    q, s = new_quantised(*x.shape)
    qb.qb_fp4_quantize(x.to(G.DEV), q, s)
    torch.cuda.synchronize()
    return q, s, values(q, s)


def near(got, a, b, n):
    """got [i, j] against sum_k a[i, k] b[j, k] (on the GPU in float64)."""
    a, b = torch.from_numpy(a).to(G.DEV), torch.from_numpy(b).to(G.DEV)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    off = (got.double() - ref).abs() - (HALF * ref.abs() + n * STEP * mag)
    assert not torch.isnan(got).any() and off.max().item() <= 0, f"{(off > 0).sum().item()} of {off.numel()} off"


# sizes on both sides of each kind of kernel, odd ones, single rows and columns
@pytest.mark.parametrize("M,N,C", [(1, 1, 1), (1, 16, 128), (1, 4096, 1024), (5, 33, 300), (16, 17, 2000), (17, 256, 640),
                                   (33, 130, 129), (64, 200, 512), (65, 129, 700), (200, 700, 130), (777, 2005, 1001),
                                   (129, 1, 4096), (3000, 4100, 260), (4000, 4096, 1300)])
def test_product(M, N, C):
    rng = np.random.default_rng(M + N + C)
    G.say(f"4-bit product M={M} N={N} C={C}")
    xq, xs, x = quantised(data(rng, M, C))
    wq, ws, w = weight(rng, N, C)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=G.DEV)
    qb.qb_fp4_product(xq, xs, wq, ws, y)
    torch.cuda.synchronize()
    near(y, x, w, C)


def test_sums_that_cancel():
    """Large products that cancel beside small ones, in one block, in blocks of
    one instruction and of different ones: the small ones' sum is left, exactly."""
    M, N, C = 48, 80, 1024
    rng = np.random.default_rng(1)
    G.say("4-bit sums that cancel")
    for first, second in ((0, 1), (0, 40), (5, 700), (130, 900), (64, 96)):
        x, w = np.zeros((M, C)), np.zeros((N, C))
        x[:, :] = rng.integers(-2, 3, (M, C)) * 2.0 ** -9
        w[:, :] = rng.integers(-2, 3, (N, C)) * 0.5
        big = 2.0 ** 9
        for c in (first, second):                      # a block of its own, whose scale holds the large value
            x[:, c // 32 * 32:c // 32 * 32 + 32] = 0
        for c, sign in ((first, 1), (second, -1)):
            x[:, c], w[:, c] = sign * big, 1.0
        (xq, xs, xv), (wq, ws) = quantised(bf16_values(x)), new_quantised(N, C)
        qb.qb_fp4_quantize_weight(G.dev(w.astype(np.float32)), wq, ws)
        y = torch.zeros((M, N), dtype=torch.bfloat16, device=G.DEV)
        qb.qb_fp4_product(xq, xs, wq, ws, y)
        torch.cuda.synchronize()
        ref = xv[:, :C] @ values(wq, ws)[:, :C].T
        mag = np.abs(xv[:, :C]) @ np.abs(values(wq, ws)[:, :C]).T
        # all terms are multiples of 2^-10 below 2^10: a sum of them in 32 bits is exact
        assert mag.max() < 2.0 ** 13 and np.array_equal(G.host(y.float()), G.host(torch.from_numpy(ref).to(torch.bfloat16).float()))


def offsets(rng, G_, M, kind, align):
    if kind == "one":                                  # everything at the last expert
        c = np.zeros(G_, np.int64)
        c[-1] = M
    else:
        w = np.exp(1.5 * rng.standard_normal(G_)) * (rng.random(G_) > 0.4)
        w[rng.integers(G_)] += 1
        c = rng.multinomial(M, w / w.sum())
    c = -(-c // align) * align
    return np.concatenate([[0], np.cumsum(c)]).astype(np.int32)


@pytest.mark.parametrize("kind", ["any", "one"])
@pytest.mark.parametrize("G_,M,N,C,align", [(1, 3, 16, 128, 1), (256, 128, 64, 520, 1), (16, 300, 130, 200, 1),
                                            (16, 700, 100, 300, 16), (7, 2000, 260, 257, 1), (32, 9000, 520, 384, 128),
                                            (256, 5000, 33, 130, 1), (3, 6000, 1024, 520, 1)])
def test_product_of_experts(G_, M, N, C, align, kind):
    rng = np.random.default_rng(G_ + M)
    off = offsets(rng, G_, M, kind, align)
    rows = int(off[-1]) + 5                            # rows past the last expert stay as they were
    G.say(f"4-bit experts' product G={G_} M={rows} N={N} C={C} align={align} {kind}")
    xq, xs, x = quantised(data(rng, rows, C))
    xs[int(off[-1]):] = 255
    wq, ws, w = weight(rng, N, C, (G_,))
    y = torch.full((rows, N), 77.0, dtype=torch.bfloat16, device=G.DEV)
    qb.qb_fp4_product(xq, xs, wq, ws, y, off=G.dev(off))
    torch.cuda.synchronize()
    for e in range(G_):
        i, j = int(off[e]), int(off[e + 1])
        if i < j:
            near(y[i:j], x[i:j], w[e], C)
    assert (y[off[-1]:] == 77.0).all()


def test_captured_and_on_another_stream():
    """A layer's step of a graph, replayed beside eager work, on a stream of its own."""
    rng = np.random.default_rng(11)
    E, N, C = 5, 130, 200
    off = offsets(rng, E, 900, "any", 1)
    R = int(off[-1])
    offd, src = G.dev(off), G.dev(rng.integers(0, 300, R).astype(np.int32))
    x, dy, w = data(rng, 300, C).to(G.DEV), data(rng, R, N).to(G.DEV), G.dev(rng.standard_normal((E, N, C)).astype(np.float32))
    (xq, xs), (dq, ds) = new_quantised(R, C), new_quantised(R, N)
    (wq, ws), (wt, wts) = new_quantised(N, C, (E,)), new_quantised(C, N, (E,))
    y = torch.zeros((R, N), dtype=torch.bfloat16, device=G.DEV)
    dx = torch.zeros((R, C), dtype=torch.bfloat16, device=G.DEV)

    def step(stream=None):
        qb.qb_fp4_quantize_weight(w, wq, ws, wt, wts, stream=stream)
        qb.qb_fp4_quantize(x, xq, xs, row_src=src, stream=stream)
        qb.qb_fp4_product(xq, xs, wq, ws, y, off=offd, stream=stream)
        qb.qb_fp4_quantize(dy, dq, ds, stream=stream)
        qb.qb_fp4_product(dq, ds, wt, wts, dx, off=offd, stream=stream)

    G.say("4-bit graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in range(4):
        x.copy_(data(rng, 300, C))
        w.mul_(1.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, wt)]
        for t in (y, dx, wt):
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        side.synchronize()
        for a, b in zip(got, (y, dx, wt)):
            assert torch.equal(a, b)
        for e in range(E):
            i, j = int(off[e]), int(off[e + 1])
            if i < j:
                near(dx[i:j], values(dq, ds)[i:j], values(wt, wts)[e], N)
