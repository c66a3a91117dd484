"""The expert layer's bias update after a batch with padding or with tokens
outside every sequence: the quantile of the live tokens' scores alone, equal
bit for bit to the oracle's over those rows; and the layer's step in a graph,
in order between its streams.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from test_gpu_expert_layer import make, test_a_training_step as training_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


class OfLiveRows:
    """The oracle over the rows that are left of `training_step`'s mask."""

    def __init__(self, oracle):
        self.oracle = oracle

    def eqb_layer(self, s, b, K):
        N = len(s)
        return self.oracle.eqb_layer(np.delete(s, slice(N // 2, N // 2 + 3), axis=0), b, K)


# the cases of the training step's own test, whose three masked rows belong to no expert's load
@pytest.mark.parametrize("N,E,K,H,M", [(300, 32, 2, 256, 200), (1000, 64, 6, 512, 130), (16, 256, 8, 256, 384)])
def test_a_training_step_with_the_update_of_its_live_rows(O, N, E, K, H, M):
    training_step(OfLiveRows(O), N, E, K, H, M)


def masks(N, kind, rng):
    """seq_off and valid of a batch, and which rows are live."""
    live = np.ones(N, bool)
    off = valid = None
    if kind in ("padding", "both", "none"):
        valid = (rng.random(N) > (1.0 if kind == "none" else 0.4)).astype(np.uint8)
        live &= valid != 0
    if kind in ("sequences", "both"):
        off = np.array([N // 7, N // 3, N // 3, N - N // 5], np.int32)
        live[:off[0]] = False
        live[off[-1]:] = False
    return off, valid, live


@pytest.mark.parametrize("kind", ["all", "padding", "sequences", "both", "none"])
@pytest.mark.parametrize("N,E,K", [(300, 32, 2), (4099, 64, 6), (70000, 256, 6), (9, 128, 15)])
def test_the_update_is_of_the_live_rows(O, N, E, K, kind):
    """Many dead rows, which hold NaN, infinities, one hidden state over and
    over, and zeros."""
    rng = np.random.default_rng(N + E)
    off, valid, live = masks(N, kind, rng)
    B = 1 if off is None else len(off) - 1
    layer, h, _ = make(N, E, K, 256, 16, B, N)
    for i, v in enumerate((float("nan"), float("inf"), 3.0, 0.0)):
        h[torch.from_numpy(np.nonzero(~live)[0][i::4]).to(G.DEV)] = v
    G.say(f"update of live rows N={N} E={E} K={K} {kind}: {live.sum()} live")
    layer.forward(h, seq_off=None if off is None else G.dev(off), valid=None if valid is None else G.dev(valid))
    torch.cuda.synchronize()
    s, b = G.host(layer.s), G.host(layer.b)
    assert layer.count.sum().item() == live.sum() * K
    for twice in range(2):
        if live.any():
            want = O.eqb_layer(s[live], b, K)
            b, keys = want["b_next"], want["key"]
        layer.update_bias()
        torch.cuda.synchronize()
        G.assert_same(f"b, update {twice}", G.host(layer.b), b)
        err = int(layer.eqb.err.item())
        if live.any():
            assert err == 0
            G.assert_same("key", G.host(layer.eqb.key), keys)
            G.assert_same("alpha", G.host(layer.alpha)[live], want["alpha"])
        else:
            assert err & 2                           # no token: the bias stays


@pytest.mark.parametrize("E,K", [(16, 3), (256, 15)])
def test_the_composed_update_leaves_rows_out(O, E, K):
    """eqb_update with topk: rows whose first choice is outside [0, E) on
    either side are not there, whatever they hold; the histogram is the live
    rows', added to what it held."""
    rng = np.random.default_rng(E)
    N = 3001
    s = (1 / (1 + np.exp(-rng.standard_normal((N, E))))).astype(np.float32)
    b = rng.uniform(-0.1, 0.1, E).astype(np.float32)
    topk = rng.integers(0, E, (N, K)).astype(np.int32)
    live = rng.random(N) < 0.7
    topk[~live, 0] = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (~live).sum())
    dirty = s.copy()
    dirty[~live] = rng.choice(np.array([np.nan, -np.inf, np.inf, 3e38], np.float32), ((~live).sum(), E))
    want = O.eqb_layer(s[live], b, K)
    G.say(f"composed update E={E} K={K}")
    sd, bd, td = G.dev(dirty), G.dev(b), G.dev(topk)
    alpha, buf = torch.empty(N, device=G.DEV), qb.EqbBuffers(1, E, device=G.DEV, lead=False)
    qb.eqb_update(sd, bd, K, alpha, buf, topk=td)
    torch.cuda.synchronize()
    assert int(buf.err.item()) == 0
    for name, got in (("hist_hi", buf.hist_hi), ("sel_hi", buf.sel_hi), ("rank_lo", buf.rank_lo),
                      ("hist_lo", buf.hist_lo), ("key", buf.key), ("q", buf.q), ("b_next", bd), ("bounds", buf.bounds)):
        G.assert_same(name, G.host(got), want[name])
    a = G.host(alpha)
    G.assert_same("alpha", a[live], want["alpha"])
    assert np.isposinf(a[~live]).all()
    got = G.host(sd)
    G.assert_same("s", got[live], s[live])
    assert not got[~live].any()
    with pytest.raises(ValueError, match="load counts every row"):
        qb.eqb_update(sd, bd, K, alpha, buf, load=torch.zeros(E, dtype=torch.int32, device=G.DEV), topk=td)


def test_the_update_balances_the_live_tokens():
    """4096 rows, 30% of them padding with one hidden state: after eight
    updates the live tokens' fullest expert has the mean load, but for the
    bf16 margins' ties and the whole ranks (a fiftieth)."""
    N, E, K = 4096, 64, 6
    layer, h, _ = make(N, E, K, 256, 16, 1, 5)
    valid = np.ones(N, np.uint8)
    valid[np.random.default_rng(5).permutation(N)[:3 * N // 10]] = 0
    valid = G.dev(valid)
    h[valid == 0] = h[0].clone()
    G.say("eight updates beside padding")
    for _ in range(8):
        layer.forward(h, valid=valid)
        layer.update_bias()
    layer.forward(h, valid=valid)
    torch.cuda.synchronize()
    load = G.host(layer.count)[0].astype(np.float64)
    assert load.sum() == G.host(valid).sum() * K
    assert load.max() / load.mean() - 1 <= 0.02, load.max() / load.mean() - 1


def test_the_step_in_a_graph_in_order():
    """Three replays of a masked step on other inputs, another layer's eager
    steps between them; each replay's results are kept before the same step
    runs eagerly on a side stream, which waits for all of it."""
    N, E, K, H, M = 200, 32, 4, 256, 130
    layer, h, dout = make(N, E, K, H, M, 1, 7)
    other, h2, dout2 = make(N, E, K, H, M, 1, 8)
    names = ("out", "loss", "dx", "dw", "dlogits", "b")
    valid = torch.ones(N, dtype=torch.uint8, device=G.DEV)
    valid[::3] = 0

    def step(l, x, d):
        l.forward(x, valid=valid)
        l.backward(d)
        l.update_bias()

    b0 = layer.b.clone()
    G.say("expert layer in a graph, in order")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(layer, h, dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layer, h, dout)
    last = None
    for k in range(3):
        g = torch.Generator(device=G.DEV).manual_seed(100 + k)
        h.copy_(torch.randn((N, H), generator=g, device=G.DEV))
        dout.copy_(torch.randn((N, M), generator=g, device=G.DEV))
        layer.b.copy_(b0)
        graph.replay()
        got = {n: getattr(layer, n).clone() for n in names}
        step(other, h2, dout2)
        layer.b.copy_(b0)
        for n in names[:-1]:
            getattr(layer, n).fill_(float("nan"))
        torch.cuda.synchronize()
        got = {n: t.float().cpu().numpy() for n, t in got.items()}
        with torch.cuda.stream(side):
            step(layer, h, dout)
        torch.cuda.synchronize()
        for n in names:
            G.assert_same(f"replay {k} {n}", got[n], getattr(layer, n).float().cpu().numpy())
        assert last is None or not np.array_equal(last, got["dw"])      # other inputs, other results
        last = got["dw"]
