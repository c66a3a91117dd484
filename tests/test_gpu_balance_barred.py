"""Experts barred by a bias of -infinity, against the same routing with the
lowest finite value in its place and against the definition in float64 (see
test_gpu_balance.py for the tolerances)."""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from test_gpu_balance import COEF, check, everything, reference, run, scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


@pytest.mark.parametrize("E,K,allowed", [(16, 4, 1), (32, 3, 20), (64, 6, 3), (64, 6, 20), (128, 15, 16), (256, 8, 0),
                                         (256, 6, 6), (256, 6, 255)])
def test_experts_barred_by_minus_infinity(E, K, allowed):
    rng = np.random.default_rng(E + allowed)
    b = np.full(E, -np.inf, np.float32)
    b[rng.permutation(E)[:allowed]] = rng.uniform(-0.1, 0.1, allowed)
    s = scores(rng, 205, E)
    G.say(f"balance barred by -inf E={E} K={K} allowed={allowed}")
    everything(s, b, K, [0, 100, 205])
    lowest = np.where(np.isinf(b), np.finfo(np.float32).min, b).astype(np.float32)
    kw = dict(off=[0, 100, 205], coef=COEF, dloss=3.0)
    got, same = run(s, b, K, **kw), run(s, lowest, K, **kw)
    for k in got:
        G.assert_same(k, got[k], same[k])


def test_experts_forced_by_infinity():
    """Two experts at +infinity come first, by index, then the largest."""
    rng = np.random.default_rng(1)
    E, K = 64, 5
    b = np.zeros(E, np.float32)
    b[[7, 40]] = np.inf
    b[3] = -np.inf
    s = scores(rng, 100, E)
    G.say("balance forced by inf")
    got = run(s, b, K, coef=COEF)
    check(got, reference(s, b, K, coef=COEF), K)
    assert (got["topk"][:, :2] == [7, 40]).all()
