"""The exchange of rows between tokens and experts (qb_dispatch, qb_combine,
qb_combine_backward) against its definition in float64.

The order is whole numbers: equal.  With u = 2^-24 and half a bf16 step 2^-8:
* out adds K products in 32 bits and is rounded once: 2^-8 |out| + 2 K u sum
  |gate row| (the second term also covers the rounding of the inexact sum);
* dgate adds H products in 32 bits: (H + 8) u sum |dout row|;
* drows is one product, rounded to 32 and to 16 bits: (2^-8 + 2 u) |drows|.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def order(topk, E, align, R):
    N, K = topk.shape
    ids = topk.reshape(-1)
    off = [0]
    pos, src = np.full(N * K, -1, np.int32), np.full(R, -1, np.int32)
    for e in range(E):
        mine = np.nonzero(ids == e)[0]
        pos[mine] = off[-1] + np.arange(len(mine))
        src[off[-1]:off[-1] + len(mine)] = mine // K
        off.append(off[-1] + -(-len(mine) // align) * align)
    return np.array(off, np.int32), src, pos.reshape(N, K)


def dispatch(topk, E, align, extra=0):
    N, K = topk.shape
    R = qb.qb_dispatch_rows(N, K, E, align) + extra
    off = torch.full((E + 1,), -7, dtype=torch.int32, device=G.DEV)
    src = torch.full((R,), -7, dtype=torch.int32, device=G.DEV)
    pos = torch.full((N, K), -7, dtype=torch.int32, device=G.DEV)
    ws = torch.full((qb.qb_dispatch_workspace_bytes(N, K, E),), 0xA5, dtype=torch.uint8, device=G.DEV)
    qb.qb_dispatch(G.dev(topk), E, align, off, src, pos, ws if ws.numel() else None)
    torch.cuda.synchronize()
    return off, src, pos, R


def experts(rng, N, K, E, kind):
    if kind == "one":                     # every token's first choice is the same expert
        ids = np.argsort(rng.random((N, E)), axis=1)[:, :K]
        ids[:, 0] = E - 1
    elif kind == "outside":               # numbers outside [0, E) go nowhere
        ids = rng.integers(-3, E + 4, (N, K))
        ids[::5] = np.int32(-2 ** 31)
    elif kind == "none":
        ids = np.full((N, K), -1)
    else:
        ids = np.argsort(rng.random((N, E)), axis=1)[:, :K]
    return ids.astype(np.int32)


@pytest.mark.parametrize("kind", ["any", "one", "outside", "none"])
@pytest.mark.parametrize("N,K,E,align", [(0, 2, 16, 128), (1, 1, 16, 1), (1, 15, 256, 128), (16, 8, 256, 1),
                                         (77, 3, 5, 7), (1024, 8, 64, 16), (1025, 8, 64, 128), (4001, 7, 255, 128),
                                         (30000, 6, 1, 3)])
def test_order(N, K, E, align, kind):
    rng = np.random.default_rng(N + E)
    if K > E and kind in ("any", "one"):
        kind = "outside"
    topk = experts(rng, N, K, E, kind)
    G.say(f"dispatch N={N} K={K} E={E} align={align} {kind}")
    off, src, pos, R = dispatch(topk, E, align, extra=3)
    ro, rs, rp = order(topk, E, align, R)
    G.assert_same("off", G.host(off), ro)
    G.assert_same("row_src", G.host(src), rs)
    G.assert_same("pos", G.host(pos), rp)


def test_order_of_many_blocks():
    """More pairs than 128 workgroups of the largest block hold."""
    rng = np.random.default_rng(3)
    N, K, E = 150000, 8, 64
    topk = rng.integers(0, E, (N, K)).astype(np.int32)
    G.say("dispatch 1.2M pairs")
    off, src, pos, R = dispatch(topk, E, 128)
    ro, rs, rp = order(topk, E, 128, R)
    G.assert_same("off", G.host(off), ro)
    G.assert_same("row_src", G.host(src), rs)
    G.assert_same("pos", G.host(pos), rp)


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).to(G.DEV)


def f64(t):
    return G.host(t.float()).astype(np.float64)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("N,K,E,H,align", [(1, 1, 16, 1, 1), (1, 8, 256, 2048, 1), (3, 15, 32, 7, 16), (64, 2, 16, 64, 1),
                                           (50, 9, 16, 65, 128), (130, 6, 64, 200, 16), (33, 8, 64, 1101, 128),
                                           (257, 4, 128, 512, 1), (20, 3, 16, 2500, 128)])
def test_combine_and_its_gradients(N, K, E, H, align, gated):
    rng = np.random.default_rng(H + N)
    topk = experts(rng, N, K, E, "any")
    topk[rng.random(N) < 0.2] = -1                       # tokens routed nowhere
    topk[rng.random((N, K)) < 0.1] = -1                  # and single choices
    G.say(f"combine N={N} K={K} E={E} H={H} align={align} gated={gated}")
    off, src, pos, R = dispatch(topk, E, align, extra=2)
    rows = bf16(rng, R, H)
    rows[src < 0] = float("nan")                         # rows of no pair reach nothing
    dout = bf16(rng, N, H)
    gate = G.dev(rng.standard_normal((N, K)).astype(np.float32)) if gated else None
    out = torch.full((N, H), 77.0, dtype=torch.bfloat16, device=G.DEV)
    drows = torch.full((R, H), 77.0, dtype=torch.bfloat16, device=G.DEV)
    dgate = torch.full((N, K), 77.0, device=G.DEV)
    qb.qb_combine(rows, pos, out, gate=gate)
    qb.qb_combine_backward(dout, rows, pos, src, drows, gate=gate, dgate=dgate)
    alone = torch.full((R, H), 77.0, dtype=torch.bfloat16, device=G.DEV)
    qb.qb_combine_backward(dout, None, pos, src, alone, gate=gate)
    torch.cuda.synchronize()
    p, r, d = G.host(pos), f64(rows), f64(dout)
    g = G.host(gate).astype(np.float64) if gated else np.ones((N, K))
    ref, mag = np.zeros((N, H)), np.zeros((N, H))
    rdr, rdg, mdg = np.zeros((R, H)), np.zeros((N, K)), np.zeros((N, K))
    for t in range(N):
        for k in range(K):
            if p[t, k] >= 0:
                one = r[p[t, k]]
                ref[t] += g[t, k] * one
                mag[t] += np.abs(g[t, k] * one)
                rdr[p[t, k]] = g[t, k] * d[t]
                rdg[t, k] = (d[t] * one).sum()
                mdg[t, k] = np.abs(d[t] * one).sum()
    assert (np.abs(f64(out) - ref) <= HALF * np.abs(ref) + 2 * K * U * mag).all()
    assert (np.abs(f64(drows) - rdr) <= (HALF + 2 * U) * np.abs(rdr)).all()
    assert (np.abs(G.host(dgate) - rdg) <= (H + 8) * U * mdg).all()
    G.assert_same("drows alone", G.host(alone.view(torch.int16)), G.host(drows.view(torch.int16)))


def test_copies_and_their_backward_are_transposes():
    """Without gates the two calls hand each expert its copy of a token and add
    the copies up again: <copies(x), r> = <x, sum(r)> on whole numbers, which
    every sum here holds exactly."""
    rng = np.random.default_rng(9)
    N, K, E, H = 200, 4, 16, 96
    topk = experts(rng, N, K, E, "any")
    G.say("exchange transposes")
    off, src, pos, R = dispatch(topk, E, 16)
    whole = lambda *s: torch.from_numpy(rng.integers(-3, 4, s).astype(np.float32)).to(torch.bfloat16).to(G.DEV)  # noqa: E731
    x, r = whole(N, H), whole(R, H)
    r[src < 0] = 0
    copies, back = torch.empty_like(r), torch.empty_like(x)
    qb.qb_combine_backward(x, None, pos, src, copies)
    qb.qb_combine(r, pos, back)
    torch.cuda.synchronize()
    assert (copies.double() * r.double()).sum().item() == (x.double() * back.double()).sum().item()
    live = src >= 0
    assert torch.equal(copies[live], x[src[live].long()]) and not copies[~live].any()


def test_graph_replays():
    """Order, sum and gradients captured once and replayed on new routes."""
    rng = np.random.default_rng(10)
    N, K, E, H = 2500, 6, 64, 128
    topk = G.dev(experts(rng, N, K, E, "any"))
    R = qb.qb_dispatch_rows(N, K, E, 128)
    i32 = dict(dtype=torch.int32, device=G.DEV)
    off, src, pos = torch.empty(E + 1, **i32), torch.empty(R, **i32), torch.empty((N, K), **i32)
    ws = torch.empty(qb.qb_dispatch_workspace_bytes(N, K, E), dtype=torch.uint8, device=G.DEV)
    assert ws.numel() > 0
    rows, dout = bf16(rng, R, H), bf16(rng, N, H)
    gate = torch.rand((N, K), device=G.DEV)
    out, drows, dgate = torch.empty_like(dout), torch.empty_like(rows), torch.empty_like(gate)

    def step():
        qb.qb_dispatch(topk, E, 128, off, src, pos, ws)
        qb.qb_combine(rows, pos, out, gate=gate)
        qb.qb_combine_backward(dout, rows, pos, src, drows, gate=gate, dgate=dgate)

    G.say("exchange graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (1, 2, 3):
        topk.copy_(G.dev(experts(np.random.default_rng(seed), N, K, E, "one")))
        graph.replay()
        torch.cuda.synchronize()
        got = [G.host(t.view(torch.int16) if t.dtype == torch.bfloat16 else t) for t in (off, src, pos, out, drows, dgate)]
        step()
        torch.cuda.synchronize()
        for a, t in zip(got, (off, src, pos, out, drows, dgate)):
            G.assert_same(f"replay {seed}", a, G.host(t.view(torch.int16) if t.dtype == torch.bfloat16 else t))


def test_the_most_tokens():
    """2^24 tokens of more than 1024 columns: 32 bits do not number their
    columns' threads.  Each token copies one row, so everything is exact but
    dgate, a sum of H products."""
    N, H, R = 1 << 24, 1032, 3
    rng = np.random.default_rng(31)
    rows = bf16(rng, R, H)
    i = torch.arange(N, dtype=torch.int32, device=G.DEV)
    pos = (i % R)[:, None].contiguous()
    out = torch.full((N, H), 7.0, dtype=torch.bfloat16, device=G.DEV)
    qb.qb_combine(rows, pos, out)
    step = 1 << 20
    for a in range(0, N, step):
        assert torch.equal(out[a:a + step], rows[pos[a:a + step, 0].long()])
    # the gradients: token t has row N - 1 - t, whose value is the token's own `out`
    back = (N - 1 - i).contiguous()
    drows = torch.full((N, H), 7.0, dtype=torch.bfloat16, device=G.DEV)
    dgate = torch.full((N, 1), 7.0, device=G.DEV)
    qb.qb_combine_backward(out, out, back[:, None].contiguous(), back, drows, dgate=dgate)
    r = rows.double().cpu()
    dots, sizes = (r @ r.T).to(G.DEV), (r.abs() @ r.abs().T).to(G.DEV)
    for a in range(0, N, step):
        mine = (i[a:a + step] % R).long()
        other = ((N - 1 - i[a:a + step]) % R).long()
        assert torch.equal(drows[a:a + step], rows[other])
        off = (dgate[a:a + step, 0].double() - dots[mine, other]).abs()
        assert bool((off <= (H + 8) * U * sizes[mine, other]).all())
    del out, drows
    torch.cuda.empty_cache()


def test_the_most_empty_rows():
    """2^30 rows, more than a launch has threads for, of which a few belong to a pair."""
    R = (1 << 30) + 77
    src = torch.full((R,), -1, dtype=torch.int32, device=G.DEV)
    kept = torch.tensor([0, 15, 16, 64, (1 << 23) - 1, 1 << 23, (1 << 29) + 5, R - 1], device=G.DEV)
    src[kept] = 0
    drows = torch.full((R, 1), 7.0, dtype=torch.bfloat16, device=G.DEV)
    none = torch.zeros(0, 1, device=G.DEV)
    qb.qb_combine_backward(none.bfloat16(), None, none.int(), src, drows)
    assert bool((drows[kept] == 7.0).all())
    drows[kept] = 0.0
    assert not bool(drows.view(torch.int16).any())
    del src, drows
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N,K,E,align", [(300001, 8, 250, 16), (2100001, 1, 3, 1)])
def test_order_of_more_blocks_than_one_adds_up(N, K, E, align):
    rng = np.random.default_rng(N)
    topk = rng.integers(-1, E + 1, (N, K)).astype(np.int32)
    off, src, pos, R = dispatch(topk, E, align, extra=5)
    ro, rs, rp = order(topk, E, align, R)
    G.assert_same("off", G.host(off), ro)
    G.assert_same("row_src", G.host(src), rs)
    G.assert_same("pos", G.host(pos), rp)
