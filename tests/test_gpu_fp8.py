"""Products in 8-bit floating point with a power-of-two scale for each block
of 128 (qb_fp8_*) against their definition in float64.

A quantised value is exact: the scale is the least power of two that keeps the
block within 448, and the value is rounded to nearest even on e4m3's grid, so
both are compared for equality.  A product of two e4m3 values is exact in 32
bits; a sum of n of them adds n terms, each addition off by at most one step,
2^-23 of the terms' magnitudes: n 2^-23 sum |a b| in 32 bits, and half a bf16
step, 2^-8 of the result, where it is rounded to bf16.  Where the caller does
not ask for exact sums, each of eight products may lose 2^-13 of the largest
of them: 8 2^-13 = 2^-10 of sum |a b| more.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu
STEP, HALF, DROP = 2.0 ** -23, 2.0 ** -8, 2.0 ** -10


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def bf16_values(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def exponent(top):
    """The least whole e >= -126 with top <= 448 * 2^e (float64, finite)."""
    e = np.full(top.shape, -126)
    for k in range(-126, 128):
        e = np.where(top > 448.0 * 2.0 ** k, k + 1, e)
    return e


def e4m3(v):
    """Nearest even on e4m3's grid: 3 fraction bits, least normal exponent -6."""
    a = np.abs(v)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -60))), -6) - 3)
    return np.rint(v / step) * step


def quantise(x):
    """x [rows, n] float64 -> the values it stands for [rows, ld], exponents [rows, blocks]."""
    rows, n = x.shape
    ld = qb.fp8_ld(n)
    t = np.zeros((rows, ld))
    t[:, :n] = x
    t = t.reshape(rows, -1, 128)
    e = exponent(np.abs(t).max(2))
    return (e4m3(t / 2.0 ** e[..., None]) * 2.0 ** e[..., None]).reshape(rows, ld), e


def values(q, s, per_row=1):
    """What e4m3 q [.., rows, ld] with scale bytes s [.., rows / per_row, sld] stands for, float64."""
    q64 = G.host(q.float()).astype(np.float64)
    e = G.host(s).astype(np.float64)[..., :q.shape[-1] // 128] - 127
    e = np.repeat(np.repeat(e, per_row, -2)[..., :q.shape[-2], :], 128, -1)
    return q64 * 2.0 ** e


def new_quantised(rows, n, lead=()):
    q = torch.full(lead + (rows, qb.fp8_ld(n)), 0x55, dtype=torch.uint8, device=G.DEV).view(torch.float8_e4m3fn)
    return q, torch.full(lead + (rows, qb.fp8_sld(n)), 0x55, dtype=torch.uint8, device=G.DEV)


def data(rng, M, C):
    """Rows and columns of very different sizes, zeros, values at the border
    of a scale and around e4m3's least normal."""
    x = rng.standard_normal((M, C)) * np.exp(2 * rng.standard_normal((M, 1))) * np.exp(rng.standard_normal((1, C)))
    x[rng.random((M, C)) < 0.05] = 0
    if M > 3:
        x[1] = 448.0 * 2.0 ** rng.integers(-4, 4, C)
        x[2] = 2.0 ** rng.integers(-18, 9, C)
        x[3] = 0
    return bf16_values(x)


@pytest.mark.parametrize("M,C", [(1, 1), (1, 4096), (3, 127), (5, 128), (130, 129), (777, 1001), (2100, 520)])
def test_quantising_is_exact(M, C):
    rng = np.random.default_rng(M + C)
    x = data(rng, M, C)
    x64 = x.double().numpy()
    G.say(f"quantise M={M} C={C}")
    q, s = new_quantised(M, C)
    qt, st = new_quantised(C, M)
    qb.qb_fp8_quantize(x.to(G.DEV), q, s)
    qb.qb_fp8_quantize_cols(x.to(G.DEV), qt, st)
    torch.cuda.synchronize()
    for got, sc, ref in ((q, s, quantise(x64)), (qt, st, quantise(x64.T))):
        G.assert_same("exponents", G.host(sc)[:, :got.shape[1] // 128].astype(np.int64) - 127, ref[1].astype(np.int64))
        assert np.array_equal(values(got, sc), ref[0])


def test_the_ends_of_the_range():
    """The largest bf16 values, the least ones, subnormals, and blocks that
    hold a NaN or an infinity (those values become NaN, the others keep the
    scale of the largest finite power)."""
    big = torch.finfo(torch.bfloat16).max
    x = torch.zeros((6, 256), dtype=torch.bfloat16)
    x[0, :3] = torch.tensor([big, -big, 1.0])
    x[1, :3] = torch.tensor([2.0 ** -133, 2.0 ** -126, -(2.0 ** -130)])
    x[2, 5], x[2, 6], x[2, 130] = float("inf"), 3.0, 2.0
    x[3, 7], x[3, 200] = float("nan"), -float("inf")
    x[4, ::2] = 464.0                       # 448 < 464: the next power
    x[5] = 448.0
    G.say("quantise ends")
    q, s = new_quantised(6, 256)
    qt, st = new_quantised(256, 6)
    qb.qb_fp8_quantize(x.to(G.DEV), q, s)
    qb.qb_fp8_quantize_cols(x.to(G.DEV), qt, st)
    torch.cuda.synchronize()
    x64, got = x.double().numpy(), values(q, s)
    finite = [0, 1, 4, 5]
    assert np.array_equal(got[finite], quantise(x64[finite])[0])
    lost = ~np.isfinite(x64)
    assert np.isnan(got[lost]).all() and not np.isnan(got[~lost]).any()
    gt = values(qt, st)
    assert np.isnan(gt[:, :6].T[lost]).all() and not np.isnan(gt[:, :6].T[~lost]).any()


def test_rows_by_number():
    """row_src: each row taken from another one, zeros outside [0, Mx)."""
    rng = np.random.default_rng(3)
    Mx, M, C = 90, 300, 333
    x = data(rng, Mx, C)
    src = rng.integers(-2, Mx + 2, M).astype(np.int32)
    picked = np.where(((src >= 0) & (src < Mx))[:, None], x.double().numpy()[np.clip(src, 0, Mx - 1)], 0)
    G.say("quantise by row number")
    q, s = new_quantised(M, C)
    qt, st = new_quantised(C, M)
    qb.qb_fp8_quantize(x.to(G.DEV), q, s, row_src=G.dev(src))
    qb.qb_fp8_quantize_cols(x.to(G.DEV), qt, st, row_src=G.dev(src))
    torch.cuda.synchronize()
    assert np.array_equal(values(q, s), quantise(picked)[0])
    assert np.array_equal(values(qt, st), quantise(picked.T)[0])


@pytest.mark.parametrize("lead,N,C", [((), 1, 1), ((), 130, 700), ((3,), 257, 128), ((2,), 64, 1030)])
def test_weights_in_both_orders(lead, N, C):
    rng = np.random.default_rng(N + C)
    w = (rng.standard_normal(lead + (N, C)) * np.exp(2 * rng.standard_normal(lead + (N, 1)))).astype(np.float32)
    G.say(f"quantise weight {lead} {N} {C}")
    q, _ = new_quantised(N, C, lead)
    qt, _ = new_quantised(C, N, lead)
    s = torch.zeros(lead + (-(-N // 128), qb.fp8_sld(C)), dtype=torch.uint8, device=G.DEV)
    st = torch.zeros(lead + (-(-C // 128), qb.fp8_sld(N)), dtype=torch.uint8, device=G.DEV)
    qb.qb_fp8_quantize_weight(G.dev(w), q, s, qt, st)
    alone, sa = new_quantised(N, C, lead)[0], torch.zeros_like(s)
    qb.qb_fp8_quantize_weight(G.dev(w), alone, sa)
    torch.cuda.synchronize()
    got, gt = values(q, s, 128), values(qt, st, 128)
    assert torch.equal(alone.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s, sa)
    assert np.array_equal(got[..., :C], np.swapaxes(gt[..., :N], -1, -2))
    assert not got[..., C:].any() and not gt[..., N:].any()
    w64 = w.astype(np.float64)
    for g in np.ndindex(*lead):
        for i in range(0, N, 128):
            for j in range(0, C, 128):
                t = w64[g][i:i + 128, j:j + 128]
                e = exponent(np.abs(t).max())
                assert int(s[g][i // 128, j // 128]) - 127 == e
                assert np.array_equal(got[g][i:i + 128, j:min(j + 128, C)], e4m3(t / 2.0 ** e) * 2.0 ** e)


def weight(rng, N, C, lead=()):
    """A laid out weight and its float64 values."""
    w = rng.standard_normal(lead + (N, C)) * np.exp(rng.standard_normal(lead + (N, 1))) / np.sqrt(C)
    q, _ = new_quantised(N, C, lead)
    s = torch.full(lead + (-(-N // 128), qb.fp8_sld(C)), 0x55, dtype=torch.uint8, device=G.DEV)
    qb.qb_fp8_quantize_weight(G.dev(w.astype(np.float32)), q, s)
    torch.cuda.synchronize()
    return q, s, values(q, s, 128)


def quantised(x):
    q, s = new_quantised(*x.shape)
    qb.qb_fp8_quantize(x.to(G.DEV), q, s)
    torch.cuda.synchronize()
    return q, s, values(q, s)


def quantised_cols(x):
    q, s = new_quantised(x.shape[1], x.shape[0])
    qb.qb_fp8_quantize_cols(x.to(G.DEV), q, s)
    torch.cuda.synchronize()
    return q, s, values(q, s)


def near(got, a, b, n, half, drop=0.0):
    """got [i, j] against sum_k a[i, k] b[j, k] (on the GPU in float64)."""
    a, b = torch.from_numpy(a).to(G.DEV), torch.from_numpy(b).to(G.DEV)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    off = (got.double() - ref).abs() - (half * ref.abs() + (n * STEP + drop) * mag)
    assert not torch.isnan(got).any() and off.max().item() <= 0, f"{(off > 0).sum().item()} of {off.numel()} off"


# sizes on both sides of each kind of kernel, odd ones, single rows and columns
@pytest.mark.parametrize("M,N,C", [(1, 1, 1), (1, 16, 128), (1, 4096, 1024), (5, 33, 300), (16, 17, 2000), (17, 256, 640),
                                   (33, 130, 129), (64, 200, 512), (65, 129, 700), (200, 700, 130), (777, 2005, 1001),
                                   (129, 1, 4096), (3000, 4100, 260)])
def test_product(M, N, C):
    rng = np.random.default_rng(M + N + C)
    G.say(f"product M={M} N={N} C={C}")
    xq, xs, x = quantised(data(rng, M, C))
    wq, ws, w = weight(rng, N, C)
    for exact in (True, False):
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=G.DEV)
        qb.qb_fp8_product(xq, xs, wq, ws, y, exact=exact)
        torch.cuda.synchronize()
        near(y, x, w, C, HALF, 0.0 if exact else DROP)


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
                                            (256, 5000, 33, 130, 1)])
def test_product_of_experts(G_, M, N, C, align, kind):
    rng = np.random.default_rng(G_ + M)
    off = offsets(rng, G_, M, kind, align)
    rows = int(off[-1]) + 5                            # rows past the last expert stay as they were
    G.say(f"experts' product G={G_} M={rows} N={N} C={C} align={align} {kind}")
    xq, xs, x = quantised(data(rng, rows, C))
    wq, ws, w = weight(rng, N, C, (G_,))
    for exact in (True, False):
        y = torch.full((rows, N), 77.0, dtype=torch.bfloat16, device=G.DEV)
        qb.qb_fp8_product(xq, xs, wq, ws, y, off=G.dev(off), exact=exact)
        torch.cuda.synchronize()
        for e in range(G_):
            i, j = int(off[e]), int(off[e + 1])
            if i < j:
                near(y[i:j], x[i:j], w[e], C, HALF, 0.0 if exact else DROP)
        assert (y[off[-1]:] == 77.0).all()


@pytest.mark.parametrize("M,N,C", [(1, 1, 1), (5, 16, 700), (128, 130, 65), (777, 505, 301), (640, 2100, 1030),
                                   (2000, 3, 4097)])
def test_weight_gradient(M, N, C):
    rng = np.random.default_rng(M + N + C)
    G.say(f"weight gradient M={M} N={N} C={C}")
    dq, ds, d = quantised_cols(data(rng, M, N))
    xq, xs, x = quantised_cols(data(rng, M, C))
    dw = torch.full((N, C), float("nan"), device=G.DEV)
    qb.qb_fp8_weight_grad(dq, ds, xq, xs, dw)
    torch.cuda.synchronize()
    near(dw, d, x, M, 0.0)


@pytest.mark.parametrize("G_,M,N,C,kind", [(1, 100, 30, 20, "any"), (16, 1999, 130, 163, "any"), (16, 1000, 64, 64, "one"),
                                           (256, 3000, 20, 30, "any"), (32, 4000, 520, 300, "any")])
def test_weight_gradient_of_experts(G_, M, N, C, kind):
    rng = np.random.default_rng(G_ + M + N)
    off = offsets(rng, G_, M, kind, 128)
    rows = int(off[-1])
    G.say(f"experts' weight gradient G={G_} M={rows} N={N} C={C} {kind}")
    dq, ds, d = quantised_cols(data(rng, rows, N))
    xq, xs, x = quantised_cols(data(rng, rows, C))
    dw = torch.full((G_, N, C), float("nan"), device=G.DEV)
    qb.qb_fp8_weight_grad(dq, ds, xq, xs, dw, off=G.dev(off))
    torch.cuda.synchronize()
    for e in range(G_):
        i, j = int(off[e]), int(off[e + 1])
        near(dw[e], d[:, i:j], x[:, i:j], j - i, 0.0)


def test_nothing_to_do():
    """No rows: nothing is read or written, and the weight gradient is zero."""
    G.say("no rows")
    xq, xs = new_quantised(0, 100)
    qb.qb_fp8_quantize(torch.empty((0, 100), dtype=torch.bfloat16, device=G.DEV), xq, xs)
    wq, ws, _ = weight(np.random.default_rng(0), 20, 100, (2,))
    off = torch.zeros(3, dtype=torch.int32, device=G.DEV)
    qb.qb_fp8_product(xq, xs, wq, ws, torch.empty((0, 20), dtype=torch.bfloat16, device=G.DEV), off=off)
    dq, ds = new_quantised(20, 0)
    xt, xts = new_quantised(100, 0)
    dw = torch.full((2, 20, 100), 77.0, device=G.DEV)
    qb.qb_fp8_weight_grad(dq, ds, xt, xts, dw, off=off)
    torch.cuda.synchronize()
    assert not dw.any()
    # every expert empty, rows that belong to none
    x = data(np.random.default_rng(1), 300, 100)
    q, s, _ = quantised(x)
    y = torch.full((300, 20), 77.0, dtype=torch.bfloat16, device=G.DEV)
    qb.qb_fp8_product(q, s, wq, ws, y, off=off)
    torch.cuda.synchronize()
    assert (y == 77.0).all()


def test_nan_stays_in_its_row():
    rng = np.random.default_rng(2)
    x = data(rng, 200, 300)
    x[100, 250] = float("nan")
    xq, xs, _ = quantised(x)
    wq, ws, _ = weight(rng, 150, 300)
    y = torch.zeros((200, 150), dtype=torch.bfloat16, device=G.DEV)
    G.say("NaN row")
    qb.qb_fp8_product(xq, xs, wq, ws, y)
    torch.cuda.synchronize()
    bad = torch.isnan(y)
    assert bad[100].all() and int(bad.sum()) == 150


def test_graph_replays():
    """Quantising, product and gradient captured once and replayed on new
    inputs, eager work between the replays."""
    rng = np.random.default_rng(4)
    M, N, C = 600, 384, 256
    x, dy = data(rng, M, C).to(G.DEV), data(rng, M, N).to(G.DEV)
    wq, ws, _ = weight(rng, N, C)
    (xq, xs), (xt, xts), (dt, dts) = new_quantised(M, C), new_quantised(C, M), new_quantised(N, M)
    y, dw = torch.empty((M, N), dtype=torch.bfloat16, device=G.DEV), torch.empty((N, C), device=G.DEV)

    def step():
        qb.qb_fp8_quantize(x, xq, xs)
        qb.qb_fp8_product(xq, xs, wq, ws, y)
        qb.qb_fp8_quantize_cols(x, xt, xts)
        qb.qb_fp8_quantize_cols(dy, dt, dts)
        qb.qb_fp8_weight_grad(dt, dts, xt, xts, dw)

    G.say("fp8 graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (1, 2, 3):
        x.copy_(data(np.random.default_rng(seed), M, C))
        graph.replay()
        torch.cuda.synchronize()
        a, b = y.clone(), dw.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), y.view(torch.int16)) and torch.equal(a, y) and torch.equal(b, dw)


# many tiles a workgroup: 128 x 128 and 256 x 256 ones, with partial tiles at both ends
@pytest.mark.parametrize("M,N,C", [(4097, 3000, 130), (4090, 4090, 384), (8101, 8190, 300)])
def test_product_of_many_tiles(M, N, C):
    rng = np.random.default_rng(M)
    G.say(f"product of many tiles M={M} N={N} C={C}")
    xq, xs, x = quantised(data(rng, M, C))
    wq, ws, w = weight(rng, N, C)
    for exact in (True, False):
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=G.DEV)
        qb.qb_fp8_product(xq, xs, wq, ws, y, exact=exact)
        torch.cuda.synchronize()
        near(y, x, w, C, HALF, 0.0 if exact else DROP)


@pytest.mark.parametrize("kind", ["any", "one"])
@pytest.mark.parametrize("N,C,align", [(2047, 257, 1), (2047, 640, 128), (700, 130, 128)])
def test_experts_of_many_tiles(N, C, align, kind):
    rng = np.random.default_rng(N + C)
    G_, M = 16, 20000
    off = offsets(rng, G_, M, kind, align)
    rows = int(off[-1]) + 3
    G.say(f"experts of many tiles N={N} C={C} align={align} {kind}")
    xq, xs, x = quantised(data(rng, rows, C))
    wq, ws, w = weight(rng, N, C, (G_,))
    y = torch.full((rows, N), 77.0, dtype=torch.bfloat16, device=G.DEV)
    qb.qb_fp8_product(xq, xs, wq, ws, y, off=G.dev(off))
    torch.cuda.synchronize()
    for e in range(G_):
        i, j = int(off[e]), int(off[e + 1])
        if i < j:
            near(y[i:j], x[i:j], w[e], C, HALF, DROP)
    assert (y[off[-1]:] == 77.0).all()


@pytest.mark.parametrize("G_,M,N,C,kind", [(0, 300, 4000, 4100, ""), (0, 700, 4093, 4090, ""),
                                           (16, 3000, 1000, 2000, "any"), (16, 3000, 700, 1163, "any"),
                                           (16, 2000, 1000, 2000, "one")])
def test_weight_gradient_of_many_tiles(G_, M, N, C, kind):
    rng = np.random.default_rng(N + C)
    off = offsets(rng, G_, M, kind, 128) if G_ else np.array([0, M])
    rows = int(off[-1])
    G.say(f"weight gradient of many tiles G={G_} M={rows} N={N} C={C} {kind}")
    dq, ds, d = quantised_cols(data(rng, rows, N))
    xq, xs, x = quantised_cols(data(rng, rows, C))
    dw = torch.full(((G_,) if G_ else ()) + (N, C), float("nan"), device=G.DEV)
    qb.qb_fp8_weight_grad(dq, ds, xq, xs, dw, off=G.dev(off) if G_ else None)
    torch.cuda.synchronize()
    for e in range(max(G_, 1)):
        i, j = int(off[e]), int(off[e + 1])
        near(dw[e] if G_ else dw, d[:, i:j], x[:, i:j], j - i, 0.0)
