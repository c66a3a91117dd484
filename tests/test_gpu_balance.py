"""Routing with a sequence-wise balance loss (qb_balance_forward / backward)
against its definition in float64.

Whole numbers (experts, counts) are equal.  With u = 2^-24 (half a step of
float32, relative):
* a gate is a quotient by a sum of K scores (K - 1 additions, a reciprocal, a
  product): (K + 2) u relative;
* a row's sum z adds at most 8 quads in sequence and 5 levels: 13 u; p = s / z
  adds a reciprocal and a product, its sum over rows 4 additions in a lane (a
  chunk of 128 rows, 32 at a time) and 6 levels; the rest is in 64 bits: every
  term is positive, so the loss is within 32 u relative;
* weight is rounded once: u relative (twice, with the 64-bit quotients: 2 u);
* dlogits: every factor of the two terms carries at most 13 + 8 roundings, and
  the differences are of the terms' magnitudes: 40 u of
  (|dloss| (|w| + sum |w| p) / z + (|g| + sum |g| gate) / total) s (1 - s).
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def reference(s, b, K, off=None, valid=None, coef=0.0, dloss=None, dgate=None):
    """The definition, row by row of the order, in float64 (numpy)."""
    N, E = s.shape
    v = s + b                                             # float32: the order is that of these sums
    order = np.lexsort((np.broadcast_to(np.arange(E), (N, E)), -v), axis=1)[:, :K]
    live = np.zeros(N, bool)
    bounds = [0, N] if off is None else [int(x) for x in off]
    live[bounds[0]:bounds[-1]] = True
    if valid is not None:
        live &= valid != 0
    s = np.where(live[:, None], s, np.float32(0.5)).astype(np.float64)
    chosen = np.take_along_axis(s, order, 1)
    total = chosen.sum(1, keepdims=True)
    ok = total > 0
    gate = np.where(ok & live[:, None], chosen / np.where(ok, total, 1), 0.0)
    z = s.sum(1, keepdims=True)
    zok = z > 0
    p = np.where(zok & live[:, None], s / np.where(zok, z, 1), 0.0)
    member = np.zeros((N, E))
    np.put_along_axis(member, order, 1.0, 1)
    member *= live[:, None]
    B = len(bounds) - 1
    spans = list(zip(bounds, bounds[1:]))
    n = sum(bool(live[i:j].any()) for i, j in spans)
    count, weight, loss = np.zeros((B, E), np.int32), np.zeros((B, E)), 0.0
    ds, size = np.zeros((N, E)), np.zeros((N, E))
    for q, (i, j) in enumerate(spans):
        T = int(live[i:j].sum())
        if T == 0:
            continue
        c = member[i:j].sum(0)
        count[q] = c
        f = c * E / (K * T)
        weight[q] = coef * (f - 1) / (n * T)
        loss += coef / n * (f * p[i:j].sum(0) / T).sum()
        if dloss is not None:
            zz = np.where(zok[i:j], z[i:j], 1)
            w = weight[q] * dloss
            on = live[i:j, None] & zok[i:j]
            ds[i:j] += np.where(on, (w - (p[i:j] @ w)[:, None]) / zz, 0)
            size[i:j] += np.where(on, (np.abs(w) + (p[i:j] @ np.abs(w))[:, None]) / zz, 0)
    if dgate is not None:
        dg = dgate.astype(np.float64)
        t = np.where(ok, total, 1)
        on = live[:, None] & ok
        add = np.where(on, (dg - (dg * gate).sum(1, keepdims=True)) / t, 0)
        mag = np.where(on, (np.abs(dg) + (np.abs(dg) * gate).sum(1, keepdims=True)) / t, 0)
        for k in range(K):
            np.put_along_axis(ds, order[:, k:k + 1], np.take_along_axis(ds, order[:, k:k + 1], 1) + add[:, k:k + 1], 1)
            np.put_along_axis(size, order[:, k:k + 1], np.take_along_axis(size, order[:, k:k + 1], 1) + mag[:, k:k + 1], 1)
    jac = s * (1 - s)
    return dict(topk=np.where(live[:, None], order, -1).astype(np.int32), gate=gate, count=count, weight=weight,
                loss=loss, dlogits=ds * jac, size=size * jac)


def run(s, b, K, off=None, valid=None, coef=0.0, dloss=None, dgate=None, stats=True):
    N, E = s.shape
    sd, bd = G.dev(s), G.dev(b)
    od = None if off is None else G.dev(np.asarray(off, np.int32))
    vd = None if valid is None else G.dev(valid)
    B = 1 if off is None else len(off) - 1
    topk = torch.full((N, K), 77, dtype=torch.int32, device=G.DEV)
    gate = torch.full((N, K), 77.0, device=G.DEV)
    out = dict(topk=topk, gate=gate)
    if stats:
        out |= dict(count=torch.full((B, E), 77, dtype=torch.int32, device=G.DEV),
                    weight=torch.full((B, E), 77.0, device=G.DEV), loss=torch.full((1,), 77.0, device=G.DEV))
        ws = torch.full((qb.qb_balance_workspace_bytes(N, E, B),), 0xA5, dtype=torch.uint8, device=G.DEV)
        qb.qb_balance_forward(sd, bd, K, topk, gate=gate, count=out["count"], weight=out["weight"], loss=out["loss"],
                              ws=ws, coef=coef, seq_off=od, valid=vd)
    else:
        qb.qb_balance_forward(sd, bd, K, topk, gate=gate, seq_off=od, valid=vd)
    if dgate is not None or dloss is not None:
        out["dlogits"] = torch.full((N, E), 77.0, device=G.DEV)
        qb.qb_balance_backward(sd, topk, weight=out["weight"] if dloss is not None else None,
                               dloss=None if dloss is None else torch.tensor([dloss], dtype=torch.float32, device=G.DEV),
                               dgate=None if dgate is None else G.dev(dgate), dlogits=out["dlogits"], seq_off=od,
                               valid=vd)
    torch.cuda.synchronize()
    return {k: G.host(v) for k, v in out.items()}


def check(got, ref, K):
    G.assert_same("topk", got["topk"], ref["topk"])
    assert (np.abs(got["gate"] - ref["gate"]) <= (K + 2) * U * ref["gate"]).all()
    if "count" in got:
        G.assert_same("count", got["count"], ref["count"])
        assert (np.abs(got["weight"] - ref["weight"]) <= 2 * U * np.abs(ref["weight"])).all()
        assert abs(float(got["loss"][0]) - ref["loss"]) <= 32 * U * abs(ref["loss"])
    if "dlogits" in got:
        bad = np.abs(got["dlogits"] - ref["dlogits"]) > 40 * U * ref["size"]
        assert not bad.any(), f"{bad.sum()} gradients off"


def scores(rng, N, E):
    return (1 / (1 + np.exp(-(rng.standard_normal((N, E)) + 0.5 * rng.standard_normal((1, E)))))).astype(np.float32)


COEF, DLOSS = float(np.float32(1e-2)), 512.0


def everything(s, b, K, off=None, valid=None, seed=0):
    rng = np.random.default_rng(seed)
    dg = (1e-3 * rng.standard_normal((s.shape[0], K))).astype(np.float32)
    kw = dict(off=off, valid=valid, coef=COEF, dloss=DLOSS, dgate=dg)
    check(run(s, b, K, **kw), reference(s, b, K, **kw), K)


@pytest.mark.parametrize("E", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("N,K", [(1, 1), (2, 15), (33, 4), (257, 5), (1000, 8), (129, 9)])
def test_one_sequence(E, N, K):
    rng = np.random.default_rng(E + N)
    G.say(f"balance N={N} E={E} K={K}")
    everything(scores(rng, N, E), rng.uniform(-0.1, 0.1, E).astype(np.float32), K)


@pytest.mark.parametrize("N,E,K,off", [
    (100, 64, 6, [0, 0, 1, 1, 40, 99, 100, 100]),          # empty ones, one token, both ends
    (100, 256, 6, [3, 40, 41, 90]),                        # rows before the first and past the last
    (5003, 64, 6, None), (40000, 128, 7, None), (700, 16, 3, list(range(0, 257)) + [700]),
    (64, 32, 2, [0] * 9),                                  # no token in any sequence
])
@pytest.mark.parametrize("masked", [False, True])
def test_sequences(N, E, K, off, masked):
    rng = np.random.default_rng(N + E)
    if off is None:
        off = [0] + sorted(int(x) for x in rng.integers(0, N + 1, 40)) + [N]
    valid = None
    if masked:
        valid = (rng.random(N) > 0.3).astype(np.uint8)
        valid[off[-2]:off[-1]] = 0                         # a sequence of padding alone
    G.say(f"balance sequences N={N} E={E} K={K} B={len(off) - 1} masked={masked}")
    s = scores(rng, N, E)
    everything(s, rng.uniform(-0.1, 0.1, E).astype(np.float32), K, off, valid)


@pytest.mark.parametrize("E,K", [(16, 3), (64, 8), (256, 6), (256, 15)])
def test_equal_values_take_the_lower_index(E, K):
    """Scores on a coarse grid: ties inside and at the end of the K largest in
    almost every row; all scores equal in some, saturated 0 and 1 in others."""
    rng = np.random.default_rng(E)
    N = 517
    s = (np.round(scores(rng, N, E) * 8) / 8).astype(np.float32)
    s[::7] = 0.5
    s[1::7] = np.where(rng.random((len(s[1::7]), E)) < 0.5, 0.0, 1.0)
    s[2::7] = 0.0
    G.say(f"balance ties E={E} K={K}")
    everything(s, np.zeros(E, np.float32), K, [0, 100, 517])


def test_dead_rows_may_hold_anything():
    """NaN, infinities and the lowest value in padded rows reach no output."""
    rng = np.random.default_rng(5)
    N, E, K = 300, 256, 6
    s = scores(rng, N, E)
    valid = (rng.random(N) > 0.4).astype(np.uint8)
    b = rng.uniform(-0.1, 0.1, E).astype(np.float32)
    dg = rng.standard_normal((N, K)).astype(np.float32)
    kw = dict(off=[0, 120, 290], valid=valid, coef=COEF, dloss=DLOSS)
    dead = np.ones(N, bool)
    dead[:290] = valid[:290] == 0
    G.say("balance dead rows")
    clean = run(s, b, K, dgate=dg, **kw)
    dirty, ddg = s.copy(), dg.copy()
    dirty[dead] = np.resize(np.array([np.nan, np.inf, -np.inf, np.finfo(np.float32).min], np.float32), (dead.sum(), E))
    ddg[dead] = np.nan
    got = run(dirty, b, K, dgate=ddg, **kw)
    for k in clean:
        G.assert_same(k, got[k], clean[k])
    assert not got["dlogits"][dead].any() and (got["topk"][dead] == -1).all()


def test_each_part_alone_and_the_same_twice():
    """Experts and gates without the loss, each output without the others, and
    every word the same on a second run."""
    rng = np.random.default_rng(6)
    N, E, K = 3000, 128, 5
    s, b = scores(rng, N, E), np.zeros(E, np.float32)
    off = [0, 1000, 1001, 3000]
    dg = rng.standard_normal((N, K)).astype(np.float32)
    G.say("balance parts")
    full = run(s, b, K, off, coef=COEF, dloss=DLOSS, dgate=dg)
    again = run(s, b, K, off, coef=COEF, dloss=DLOSS, dgate=dg)
    for k in full:
        G.assert_same(k, again[k], full[k])
    alone = run(s, b, K, off, stats=False)
    G.assert_same("topk", alone["topk"], full["topk"])
    G.assert_same("gate", alone["gate"], full["gate"])
    for kw in (dict(dloss=DLOSS), dict(dgate=dg)):
        ref = reference(s, b, K, off, coef=COEF, **kw)
        check(run(s, b, K, off, coef=COEF, **kw), ref, K)
    ws = torch.empty(qb.qb_balance_workspace_bytes(N, E, 1), dtype=torch.uint8, device=G.DEV)
    loss = torch.empty(1, device=G.DEV)
    topk = torch.empty((N, K), dtype=torch.int32, device=G.DEV)
    qb.qb_balance_forward(G.dev(s), G.dev(b), K, topk, loss=loss, ws=ws, coef=COEF)
    ref = reference(s, b, K, coef=COEF)
    assert abs(float(loss.item()) - ref["loss"]) <= 32 * U * ref["loss"]


def test_gradient_is_the_slope():
    """Against differences of the definition in float64, the counts held: a
    step of h in one logit changes it by h times its gradient to O(h^2)."""
    rng = np.random.default_rng(7)
    N, E, K = 12, 16, 3
    logits = rng.standard_normal((N, E))
    b = rng.uniform(-0.1, 0.1, E)
    off = [0, 5, 12]
    dg = rng.standard_normal((N, K)).astype(np.float32)
    s32 = (1 / (1 + np.exp(-logits))).astype(np.float32)
    ref = reference(s32, b.astype(np.float32), K, off, coef=COEF)
    logits = np.log(s32.astype(np.float64) / (1 - s32.astype(np.float64)))

    def value(x):
        s = 1 / (1 + np.exp(-x))
        p = s / s.sum(1, keepdims=True)
        total = 0.0
        for q, (i, j) in enumerate(zip(off, off[1:])):
            T = j - i
            total += DLOSS * COEF / 2 * (ref["count"][q] * E / (K * T) * p[i:j].sum(0) / T).sum()
        ch = np.take_along_axis(s, ref["topk"].astype(np.int64), 1)
        return total + (dg * ch / ch.sum(1, keepdims=True)).sum()

    G.say("balance differences")
    got = run(s32, b.astype(np.float32), K, off, coef=COEF, dloss=DLOSS, dgate=dg)["dlogits"]
    h = 1e-5
    for i, e in [(0, 0), (0, int(ref["topk"][0, 0])), (4, 7), (5, int(ref["topk"][5, 2])), (11, 15)]:
        up, dn = logits.copy(), logits.copy()
        up[i, e] += h
        dn[i, e] -= h
        slope = (value(up) - value(dn)) / (2 * h)
        assert abs(got[i, e] - slope) <= 1e-6 * max(1.0, np.abs(got).max())


def test_graph_replays_on_another_stream():
    """Captured on a side stream and replayed on new scores, with eager work
    between the replays."""
    rng = np.random.default_rng(8)
    N, E, K = 2000, 64, 6
    off = torch.tensor([0, 700, 2000], dtype=torch.int32, device=G.DEV)
    s = G.dev(scores(rng, N, E))
    b = torch.zeros(E, device=G.DEV)
    mk = lambda *sh, dt=torch.float32: torch.empty(sh, dtype=dt, device=G.DEV)  # noqa: E731
    topk, gate, count, weight, loss = mk(N, K, dt=torch.int32), mk(N, K), mk(2, E, dt=torch.int32), mk(2, E), mk(1)
    dg, dx = torch.ones((N, K), device=G.DEV), mk(N, E)
    ws = mk(qb.qb_balance_workspace_bytes(N, E, 2), dt=torch.uint8)

    def step():
        qb.qb_balance_forward(s, b, K, topk, gate=gate, count=count, weight=weight, loss=loss, ws=ws, coef=COEF,
                              seq_off=off)
        qb.qb_balance_backward(s, topk, weight=weight, dgate=dg, dlogits=dx, seq_off=off)

    G.say("balance graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (1, 2, 3):
        s.copy_(G.dev(scores(np.random.default_rng(seed), N, E)))
        graph.replay()
        torch.cuda.synchronize()
        got = [G.host(t) for t in (topk, gate, count, weight, loss, dx)]
        step()
        torch.cuda.synchronize()
        for name, a, t in zip(("topk", "gate", "count", "weight", "loss", "dlogits"), got,
                              (topk, gate, count, weight, loss, dx)):
            G.assert_same(f"replay {seed} {name}", a, G.host(t))


@pytest.mark.parametrize("E,K", [(16, 3), (32, 8), (64, 7), (128, 15), (256, 1), (256, 6), (256, 8), (256, 15)])
def test_values_that_differ_in_their_last_bits(E, K):
    """Every row's scores lie within 64 float32 steps of each other, so the
    order is decided below any coarser key; half of the rows are separated
    again by the bias."""
    rng = np.random.default_rng(E + K)
    N = 301
    s = (0.5 + 2.0 ** -24 * rng.integers(0, 65, (N, E))).astype(np.float32)
    s[::3] -= np.float32(0.25)
    s[1::3] = (2.0 ** -140 * rng.integers(0, 9, s[1::3].shape)).astype(np.float32)    # subnormal, and zeros
    G.say(f"balance last bits E={E} K={K}")
    everything(s, np.zeros(E, np.float32), K, [0, 7, 300])
    b = np.where(rng.random(E) < 0.5, 0.25, 0.0).astype(np.float32)
    s[1::3] = scores(rng, len(s[1::3]), E)
    everything(s, b, K, [0, 7, 300])


@pytest.mark.parametrize("E,K,allowed", [(16, 4, 1), (64, 6, 3), (256, 8, 0), (256, 6, 6), (128, 15, 16)])
def test_experts_barred_by_the_lowest_value(E, K, allowed):
    """A bias of the lowest float32 bars an expert; with fewer experts left
    than K the barred ones follow by index (their sums are all that value)."""
    rng = np.random.default_rng(E + allowed)
    b = np.full(E, np.finfo(np.float32).min, np.float32)
    b[rng.permutation(E)[:allowed]] = 0.1
    G.say(f"balance barred E={E} K={K} allowed={allowed}")
    everything(scores(rng, 205, E), b, K, [0, 100, 205])


@pytest.mark.parametrize("E,K", [(32, 4), (128, 6), (256, 6)])
@pytest.mark.parametrize("N", [31, 500, 33000])
def test_short_sequences(E, K, N):
    """Sequences of one to five tokens with empty ones among them, so that one
    workgroup's rows end many; at 33,000 tokens a workgroup takes several steps."""
    rng = np.random.default_rng(E + N)
    lengths = rng.integers(0, 6, 3 * N // 10)
    off = [0] + [int(x) for x in np.minimum(np.cumsum(lengths), N)]
    off += [off[-1], N]
    valid = (rng.random(N) > 0.2).astype(np.uint8)
    G.say(f"balance short sequences N={N} E={E} B={len(off) - 1}")
    everything(scores(rng, N, E), rng.uniform(-0.1, 0.1, E).astype(np.float32), K, off, valid)
