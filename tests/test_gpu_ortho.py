"""The orthogonalised update (qb_orthogonalize) against its formula in float64.

The result is rounded to bf16: half a step, 2^-8 of its norm at most.  Inside,
values are rounded to one or two 16-bit parts where the kernels say so; what
that does to a result follows from the matrix, so ``rounded`` makes the same
roundings in float64 and the kernels may be off by twice what it is off by (they
round sums that are held in 32 bits, which changes which way single values go).
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
POLY = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def formula(x, steps=5, poly=POLY, one=lambda t, s: t, two=lambda t, s: t):
    """The definition for one matrix; one, two: roundings of values held times s in one and in two parts."""
    a, b, c = poly
    x = x.double()
    n = torch.linalg.vector_norm(x)
    if n > 0:
        x = x / n
    tall = x.shape[0] > x.shape[1]
    x = two(x.T.contiguous() if tall else x, 4096.0)
    for i in range(steps):
        rough = min(x.shape) >= 256 and i < 3 and i + 2 < steps
        r = one(x, 4096.0)
        s = two(r @ r.T, 256.0)
        q = one(s, 256.0) if rough else s
        p = (one if rough else two)(b * s + c * (q @ q), 256.0)
        x = two(a * x + p @ r, 4096.0)
    return x.T if tall else x


def rounded(x, steps=5, poly=POLY):
    def one(t, s):
        return (t * s).half().double() / s

    def two(t, s):
        hi = one(t, s)
        return hi + one(t - hi, s)

    return formula(x, steps, poly, one, two)


def orthogonalized(x, **kw):
    G_, N, C = (1,) * (3 - x.dim()) + tuple(x.shape)
    ws = torch.full((qb.qb_orthogonalize_workspace_bytes(G_, N, C),), 0xFF, dtype=torch.uint8, device=G.DEV)
    o = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device=G.DEV)
    qb.qb_orthogonalize(x, o, ws, **kw)
    torch.cuda.synchronize()
    return o


def near(o, x, **kw):
    want = formula(x, **kw)
    size = torch.linalg.vector_norm(want)
    off = torch.linalg.vector_norm(o.double() - want)
    inside = torch.linalg.vector_norm(rounded(x, **kw) - want)
    assert off <= HALF * size + 2 * inside, f"off {off / size:.2e}, rounding inside {inside / size:.2e}"
    assert inside <= 4e-3 * size


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(G.DEV)


# squares, wide and tall ones, odd sizes, sizes for every tile
SIZES = [((), 1, 1), ((), 1, 300), ((), 300, 1), ((), 2, 3), ((3,), 16, 16), ((2,), 33, 70), ((2,), 70, 33), ((5,), 301, 165),
         ((5,), 165, 301), ((1,), 128, 256), ((), 512, 1024), ((), 1024, 512), ((16,), 520, 640), ((16,), 640, 520),
         ((40,), 130, 1100), ((40,), 1100, 130), ((24,), 1024, 1030), ((24,), 1030, 1024), ((300,), 40, 24)]


@pytest.mark.parametrize("lead,N,C", SIZES)
def test_against_the_formula(lead, N, C):
    rng = np.random.default_rng(N + C)
    G.say(f"orthogonalize {lead} {N} {C}")
    x = randn(rng, *lead, N, C) * torch.exp(randn(rng, *lead, N, 1)) * 1e-3
    o = orthogonalized(x)
    for g in list(np.ndindex(*lead))[:6] + list(np.ndindex(*lead))[-1:]:
        near(o[g], x[g])


@pytest.mark.parametrize("steps,poly", [(1, POLY), (2, POLY), (10, POLY), (12, (1.5, -0.5, 0.0)), (8, (1.875, -1.25, 0.375))])
def test_steps_and_polynomials(steps, poly):
    rng = np.random.default_rng(steps)
    x = randn(rng, 2, 96, 200)
    G.say(f"orthogonalize steps={steps} poly={poly}")
    o = orthogonalized(x, steps=steps, poly=poly)
    for g in range(2):
        near(o[g], x[g], steps=steps, poly=poly)


def test_singular_values():
    """Singular values of 1/100 of the largest and more end between 0.7 and 1.2,
    the singular vectors stay."""
    rng = np.random.default_rng(4)
    u = torch.linalg.qr(randn(rng, 64, 64).double())[0]
    v = torch.linalg.qr(randn(rng, 200, 64).double())[0]
    s = torch.logspace(0, -1.3, 64, dtype=torch.float64, device=G.DEV)
    G.say("orthogonalize singular values")
    o = orthogonalized((u * s @ v.T).float()).double()
    d = u.T @ o @ v
    assert d.diagonal().min() > 0.65 and d.diagonal().max() < 1.25
    assert (d - torch.diag(d.diagonal())).abs().max() < 0.02


def test_few_directions():
    """A matrix of low rank: what is not in it stays out of the result."""
    rng = np.random.default_rng(6)
    x = randn(rng, 300, 20) @ randn(rng, 20, 500)
    G.say("orthogonalize low rank")
    o = orthogonalized(x)
    near(o, x)
    assert torch.linalg.matrix_rank(o.double(), tol=0.1) == 20


def test_zero_and_not_finite():
    rng = np.random.default_rng(8)
    x = randn(rng, 5, 40, 56)
    x[1] = 0
    x[2, 3, 5], x[3, 39, 55] = float("nan"), float("inf")
    G.say("orthogonalize zero, NaN")
    o = orthogonalized(x)
    assert (o[1] == 0).all() and torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
    near(o[0], x[0])
    near(o[4], x[4])


@pytest.mark.parametrize("size", [1e-30, 1e-42, 1e30])
def test_the_size_of_the_matrix_does_not_matter(size):
    rng = np.random.default_rng(10)
    x = (randn(rng, 30, 50).double() * size).float()
    G.say(f"orthogonalize size {size}")
    near(orthogonalized(x), x)


def test_at_any_address():
    rng = np.random.default_rng(12)
    x = randn(rng, 37, 51)
    flat = torch.empty(37 * 51 + 4, device=G.DEV)[1:1 + 37 * 51].view(37, 51)
    flat.copy_(x)
    out = torch.zeros(37 * 51 + 4, dtype=torch.bfloat16, device=G.DEV)
    o = out[3:3 + 37 * 51].view(37, 51)
    ws = torch.empty(qb.qb_orthogonalize_workspace_bytes(1, 37, 51), dtype=torch.uint8, device=G.DEV)
    G.say("orthogonalize unaligned")
    qb.qb_orthogonalize(flat, o, ws)
    torch.cuda.synchronize()
    near(o, x)
    assert (out[:3] == 0).all() and out[-1] == 0


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(14)
    x = randn(rng, 3, 72, 130)
    o = torch.zeros(x.shape, dtype=torch.bfloat16, device=G.DEV)
    ws = torch.empty(qb.qb_orthogonalize_workspace_bytes(*x.shape), dtype=torch.uint8, device=G.DEV)
    G.say("orthogonalize graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        qb.qb_orthogonalize(x, o, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qb.qb_orthogonalize(x, o, ws)
    for k in range(4):
        x.copy_(randn(rng, 3, 72, 130))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone()
        o.zero_()
        side.wait_stream(torch.cuda.current_stream())
        qb.qb_orthogonalize(x, o, ws, stream=side)
        side.synchronize()
        assert torch.equal(got, o)
        near(o[0], x[0])
