"""qb_orthogonalize holds its values in two fp16 parts throughout: its results
are the formula's but for their own rounding to bf16, by the bound of
ortho_forms.py, which test_ortho_bound_cpu.py shows to refuse any part left out.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from ortho_forms import POLY, above_rounding, bound, coarse, formula, norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(G.DEV)


def orthogonalized(x, **kw):
    g, N, C = (1,) * (3 - x.dim()) + tuple(x.shape)
    ws = torch.full((qb.qb_orthogonalize_workspace_bytes(g, N, C),), 0xFF, dtype=torch.uint8, device=G.DEV)
    o = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device=G.DEV)
    qb.qb_orthogonalize(x, o, ws, **kw)
    torch.cuda.synchronize()
    return o


def keeps(o, x, **kw):
    want = formula(x, **kw)
    off, most = above_rounding(o, want), bound(x, want, **kw)
    assert off <= most, f"above its rounding by {off / norm(want):.2e}, at most {most / norm(want):.2e}"


# wide, tall and square ones, odd sizes, sizes for every tile of each product
SIZES = [((), 1, 1), ((), 1, 300), ((), 300, 1), ((), 2, 3), ((3,), 16, 16), ((2,), 33, 70), ((2,), 70, 33), ((), 128, 256),
         ((5,), 301, 165), ((5,), 165, 301), ((), 512, 1024), ((), 1024, 512), ((16,), 520, 640), ((16,), 640, 520),
         ((24,), 1024, 1030), ((24,), 1030, 1024)]


@pytest.mark.parametrize("lead,N,C", SIZES)
def test_as_the_formula_in_32_bits(lead, N, C):
    rng = np.random.default_rng(N + 2 * C)
    G.say(f"orthogonalize exactly {lead} {N} {C}")
    x = randn(rng, *lead, N, C) * torch.exp(randn(rng, *lead, N, 1)) * 1e-3
    o = orthogonalized(x)
    for g in list(np.ndindex(*lead))[:3] + list(np.ndindex(*lead))[-1:]:
        keeps(o[g], x[g])


@pytest.mark.parametrize("steps,poly", [(1, POLY), (3, POLY), (10, POLY), (12, (1.5, -0.5, 0.0)), (8, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("N,C", [(96, 200), (300, 280)])
def test_steps_and_polynomials(N, C, steps, poly):
    rng = np.random.default_rng(steps + N)
    x = randn(rng, 2, N, C)
    G.say(f"orthogonalize exactly {N} {C} steps={steps} poly={poly}")
    o = orthogonalized(x, steps=steps, poly=poly)
    for g in range(2):
        keeps(o[g], x[g], steps=steps, poly=poly)


# sizes where roundings add up evenly, for every tile and with and without the steps of one pass
@pytest.mark.parametrize("lead,N,C", [((), 128, 256), ((5,), 301, 165), ((), 512, 1024), ((), 1024, 512), ((16,), 520, 640),
                                      ((16,), 640, 520), ((24,), 1024, 1030), ((24,), 1030, 1024)])
def test_the_coarse_form(lead, N, C):
    """The roundings inside are of the simulated size, and the result's own is independent of them: the two add up as
    squares (a quarter more inside for what single matrices differ by)."""
    rng = np.random.default_rng(N + 2 * C)
    G.say(f"orthogonalize coarsely {lead} {N} {C}")
    x = randn(rng, *lead, N, C)
    o = orthogonalized(x, exact=False)
    for g in list(np.ndindex(*lead))[:2] + list(np.ndindex(*lead))[-1:]:
        want = formula(x[g])
        own = norm(want.to(torch.bfloat16) - want)
        inside = norm(coarse(x[g]) - want)
        off = norm(o[g] - want)
        assert off ** 2 <= own ** 2 + (1.25 * inside) ** 2
        assert off ** 2 >= own ** 2 + (0.75 * inside) ** 2  # (and it is the coarse form that ran)


@pytest.mark.parametrize("lead,N,C", [((), 40, 65536), ((), 65536, 40), ((), 4096, 4096), ((2,), 8200, 2000), ((), 1500, 8200),
                                      ((), 8192, 8192)])
def test_large_matrices(lead, N, C):
    rng = np.random.default_rng(N + C)
    G.say(f"orthogonalize exactly {lead} {N} {C}")
    x = torch.randn(lead + (N, C), generator=torch.Generator(device=G.DEV).manual_seed(N + C), device=G.DEV)
    x *= torch.exp(0.5 * randn(rng, N, 1))
    o = orthogonalized(x)
    for g in np.ndindex(*lead):
        keeps(o[g], x[g])


# between them they have singular values from 1/200 of their norm to nearly all of it
@pytest.mark.parametrize("N,C,first", [(64, 200, 1.0), (64, 200, 0.2), (200, 64, 0.1), (300, 300, 0.05)])
def test_the_singular_values_that_are_promised(N, C, first):
    """1/200 of the norm and more end between 0.68 and 1.16 (and a bf16 result's
    rounding, 2^-8 of its norm in all directions together); what the vectors are stays."""
    rng = np.random.default_rng(N + C)
    R = min(N, C)
    u = torch.linalg.qr(randn(rng, N, R).double())[0]
    v = torch.linalg.qr(randn(rng, C, R).double())[0]
    s = torch.logspace(0, 0, R, dtype=torch.float64, device=G.DEV) * 0.0055
    s[0] = first
    s[1:9] = torch.logspace(-2.2, -1, 8, dtype=torch.float64, device=G.DEV)
    s /= torch.linalg.vector_norm(s)
    assert s.min() >= 1 / 200
    G.say(f"orthogonalize singular values {N} {C} {first}")
    o = orthogonalized(((u * s) @ v.T).float()).double()
    d = u.T @ o @ v
    # o's roundings, each at most 2^-8 of a value, seen along one pair of directions
    off = torch.sqrt((u.square().T @ (o * 2.0 ** -8).square()) @ v.square())
    low, high = d.diagonal() + 4 * off.diagonal(), d.diagonal() - 4 * off.diagonal()
    assert low.min() >= 0.68 and high.max() <= 1.16, (low.min().item(), high.max().item())
    assert ((d - torch.diag(d.diagonal())).abs() <= 6 * off).all()


def test_the_layer_passes_the_choice_on():
    from test_gpu_expert_layer import make

    layer, h, dout = make(200, 32, 4, 256, 256, 1, 1)
    G.say("a layer's orthogonalized update, both forms")
    layer.forward(h)
    _, dw, _ = layer.backward(dout)
    for exact in (True, False):
        o = layer.orthogonalized(exact=exact).clone()
        assert torch.equal(o, orthogonalized(dw, exact=exact))
    keeps(layer.orthogonalized()[3], dw[3])
