"""The sums of the 8-bit products where they cancel: without `exact=False` a
call holds them in 32 bits, whatever its number of rows.

The inputs are quantised without rounding and every partial sum of a product,
in any order, is a multiple of 2^-9 below 2^15, so 32 bits hold it; the result
is a multiple of 2^-9 of at most 8 bits, so bf16 holds it.  The results are
therefore equal to the definition's, with no tolerance.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def cancelling(rng, M, N, C):
    """x [M, C]: 256 and -256 in every eight columns (at the same places in all
    rows), 0 or +-2^-9 elsewhere.  w [N, C]: +-1, the same sign where x's large
    values meet it."""
    x = rng.integers(-1, 2, (M, C)) * 2.0 ** -9
    w = rng.choice([-1.0, 1.0], (N, C))
    for c in range(0, C - 7, 8):
        i, j = c + rng.permutation(8)[:2]
        x[:, i], x[:, j] = 256.0, -256.0
        w[:, j] = w[:, i]
    return x, w


def quantised(x):
    M, C = x.shape
    xq = torch.empty((M, qb.fp8_ld(C)), dtype=qb.F8, device=G.DEV)
    xs = torch.empty((M, qb.fp8_sld(C)), dtype=torch.uint8, device=G.DEV)
    qb.qb_fp8_quantize(G.dev(x.astype(np.float32)).to(torch.bfloat16), xq, xs)
    return xq, xs


def weight(w):
    N, C = w.shape[-2:]
    lead = w.shape[:-2]
    wq = torch.empty(lead + (N, qb.fp8_ld(C)), dtype=qb.F8, device=G.DEV)
    ws = torch.empty(lead + (-(-N // 128), qb.fp8_sld(C)), dtype=torch.uint8, device=G.DEV)
    qb.qb_fp8_quantize_weight(G.dev(w.astype(np.float32)), wq, ws)
    return wq, ws


# one row, the two kernels of few rows, and each kind of tile
@pytest.mark.parametrize("M,N,C", [(1, 512, 1024), (20, 300, 1000), (33, 130, 512), (300, 512, 1024),
                                   (3000, 4100, 264), (4090, 4090, 384)])
def test_a_sum_that_cancels(M, N, C):
    rng = np.random.default_rng(M + N)
    x, w = cancelling(rng, M, N, C)
    ref = x @ w.T
    assert np.abs(ref).max() <= 0.5 and (ref != 0).mean() > 0.5
    G.say(f"cancelling sums M={M} N={N} C={C}")
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=G.DEV)
    qb.qb_fp8_product(*quantised(x), *weight(w), y)
    torch.cuda.synchronize()
    wrong = G.host(y.double()) != ref
    assert not wrong.any(), f"{wrong.sum()} of {wrong.size} results lost bits"


@pytest.mark.parametrize("E,M,N,C", [(16, 40, 300, 512), (16, 700, 260, 512), (7, 9000, 1030, 264)])
def test_an_experts_sum_that_cancels(E, M, N, C):
    rng = np.random.default_rng(E + M)
    x, w = cancelling(rng, M, E * N, C)
    assert np.abs(x @ w.T).max() <= 0.5
    w = w.reshape(E, N, C)
    off = np.concatenate([[0], np.sort(rng.integers(0, M + 1, E - 1)), [M]]).astype(np.int32)
    G.say(f"cancelling sums of experts E={E} M={M} N={N} C={C}")
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=G.DEV)
    qb.qb_fp8_product(*quantised(x), *weight(w), y, off=G.dev(off))
    torch.cuda.synchronize()
    got = G.host(y.double())
    for e in range(E):
        i, j = off[e], off[e + 1]
        wrong = got[i:j] != x[i:j] @ w[e].T
        assert not wrong.any(), f"expert {e}: {wrong.sum()} of {wrong.size} results lost bits"


def test_the_layer_makes_the_callers_choice():
    """An ExpertLayer's experts' rows: sums of H terms in 32 bits, H 2^-23 of
    their magnitudes, and half a bf16 step; up to 2^-10 of the magnitudes more
    with exact=False, which is then used."""
    from test_gpu_expert_layer import close, held, make

    N, E, K, H, M = 2000, 16 * 2, 4, 512, 130
    rows = {}
    for exact in (True, False):
        layer, h, _ = make(N, E, K, H, M, 1, 3)
        assert layer.exact is True
        layer.exact = exact
        G.say(f"expert layer exact={exact}")
        layer.forward(h)
        torch.cuda.synchronize()
        x, w, start = held(layer.xq, layer.xs), held(layer.wq, layer.ws, 128), layer.off.tolist()
        for e, (i, j) in enumerate(zip(start, start[1:])):
            close("rows", layer.rows[i:j], x[i:j] @ w[e].T, x[i:j].abs() @ w[e].abs().T, H,
                  drop=0.0 if exact else 2.0 ** -10)
        rows[exact] = layer.rows[:start[-1]].clone()
    assert not torch.equal(rows[True], rows[False])
