"""The products of few rows, where a workgroup's waves share a sum out 1, 2, 4 or
8 ways and take 16 or 32 rows, and the products at the sizes of large layers.

Tolerances are those of test_gpu_bf16.py and test_gpu_fp4.py.  Which kernel ran
is read from a trace of the call.
"""
import numpy as np
import pytest
import torch

from exact_quantile_selection_amd import qb

import gpu_util as G
from test_gpu_bf16 import BF16, HALF, NAN, STEP, data, near, offsets, rows, taken
from test_gpu_fp4 import GRID

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qb.lib()


def ran(call, kernel):
    """`call` ran this kernel (where this machine gives a trace)."""
    from torch.profiler import ProfilerActivity, profile

    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    names = [e.name for e in p.events() if "qbk" in e.name]
    assert not names or any(kernel in n for n in names), names


def quantised(x):
    """x bf16 [.., rows, n], or float for weights, in 4 bits."""
    lead, (M, n) = tuple(x.shape[:-2]), x.shape[-2:]
    q = torch.full(lead + (M, qb.fp4_ld(n)), 0x55, dtype=torch.uint8, device=G.DEV)
    s = torch.full(lead + (M, qb.fp4_sld(n)), 255, dtype=torch.uint8, device=G.DEV)
    (qb.qb_fp4_quantize if x.dtype is BF16 else qb.qb_fp4_quantize_weight)(x, q, s)
    return q, s


def values(q, s):
    """What it stands for, in 64 bits."""
    grid = torch.tensor(np.concatenate([GRID, -GRID]), dtype=torch.float64, device=G.DEV)
    v = torch.stack([grid[(q & 15).long()], grid[(q >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


# rows, columns and length that give each way to share out at 256 CUs, rows of fewer than 8 values among them
FEW = [(1, 1, 3, 32768, 200), (1, 1, 4, 33001, 5), (1, 2, 3, 16384, 600), (1, 2, 3, 33000, 600), (1, 2, 2, 16390, 7),
       (1, 4, 3, 8300, 600), (1, 4, 3, 8200, 5), (1, 8, 16, 500, 2000), (2, 4, 30, 8190, 264), (2, 4, 17, 8192, 6),
       (2, 8, 32, 4096, 1111)]


@pytest.mark.parametrize("MT,KW,M,N,C", FEW)
def test_bf16(MT, KW, M, N, C):
    rng = np.random.default_rng(M + N + C)
    G.say(f"bf16 few rows M={M} N={N} C={C}")
    w = data(rng, N, C)
    for src in (None, rows(rng, M, 9)):
        x = data(rng, M if src is None else 9, C)
        y = torch.full((M, N), NAN, dtype=BF16, device=G.DEV)
        ran(lambda: qb.qb_bf16_product(x, w, y, row_src=src), f"k_bf16_thin<{MT}, {KW}, {str(C < 8).lower()}>")
        near(y, taken(x, src), w.T, HALF)


@pytest.mark.parametrize("KW,C", [(1, 200), (1, 504), (2, 520), (2, 1024)])
def test_bf16_of_experts(KW, C):
    rng = np.random.default_rng(C)
    E, N = 256, 400
    off = offsets(rng, E, 200, "any")
    R = int(off[-1]) + 3
    G.say(f"bf16 few rows of experts C={C}")
    x, w, src = data(rng, 30, C), data(rng, E, N, C), rows(rng, R, 30)
    y = torch.full((R, N), 77.0, dtype=BF16, device=G.DEV)
    ran(lambda: qb.qb_bf16_product(x, w, y, off=G.dev(off), row_src=src), f"k_bf16_thin<1, {KW}, false>")
    t = taken(x, src)
    for e in range(E):
        i, j = int(off[e]), int(off[e + 1])
        near(y[i:j], t[i:j], w[e].T, HALF)
    assert (y[off[-1]:] == 77.0).all()


def near4(y, xq, xs, wq, ws, n):
    a, b = values(xq, xs), values(wq, ws)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    off = (y.double() - ref).abs() - (HALF * ref.abs() + n * STEP * mag)
    assert not torch.isnan(y).any() and off.max().item() <= 0, f"{(off > 0).sum().item()} of {off.numel()} off"


# (a row of n values is ceil(n / 256) * 64 words long, and 512 of them begin a sum in two)
FEW4 = [(1, 1, 3, 32768, 200), (1, 1, 4, 33001, 1700), (1, 2, 3, 16384, 300), (1, 2, 3, 33000, 2000), (1, 4, 3, 8300, 600),
        (1, 8, 16, 500, 2000), (2, 4, 30, 8190, 264), (2, 8, 32, 4096, 1111)]


@pytest.mark.parametrize("MT,KW,M,N,C", FEW4)
def test_4_bits(MT, KW, M, N, C):
    rng = np.random.default_rng(M + N + C)
    G.say(f"4-bit few rows M={M} N={N} C={C}")
    (xq, xs), (wq, ws) = quantised(data(rng, M, C)), quantised(data(rng, N, C).float())
    y = torch.full((M, N), NAN, dtype=BF16, device=G.DEV)
    ran(lambda: qb.qb_fp4_product(xq, xs, wq, ws, y), f"k_fp4_thin<{MT}, {KW}>")
    near4(y, xq, xs, wq, ws, C)


@pytest.mark.parametrize("M,N,C", [(1, 4096, 14336), (50, 7168, 4096), (600, 4096, 7168), (5000, 7168, 2048)])
def test_the_sizes_of_large_layers(M, N, C):
    rng = np.random.default_rng(M + N)
    G.say(f"large layers M={M} N={N} C={C}")
    x, w, dy = data(rng, M, C), data(rng, N, C), data(rng, M, N)
    y, dx = torch.full((M, N), NAN, dtype=BF16, device=G.DEV), torch.full((M, C), NAN, dtype=BF16, device=G.DEV)
    dw = torch.full((N, C), NAN, device=G.DEV)
    qb.qb_bf16_product(x, w, y)
    qb.qb_bf16_product(dy, w, dx, transposed=True)
    qb.qb_bf16_weight_grad(dy, x, dw)
    torch.cuda.synchronize()
    near(y, x, w.T, HALF)
    near(dx, dy, w, HALF)
    near(dw, dy.T, x, 0.0)
    (xq, xs), (wq, ws) = quantised(x), quantised(w.float())
    y.fill_(NAN)
    qb.qb_fp4_product(xq, xs, wq, ws, y)
    torch.cuda.synchronize()
    near4(y, xq, xs, wq, ws, C)


@pytest.mark.parametrize("M", [3, 90])
def test_scales_far_from_one(M):
    """Blocks of the type's largest and smallest scales, whose products are ordinary numbers."""
    rng = np.random.default_rng(M)
    N, C = 100, 512
    G.say(f"4-bit scales far from one M={M}")
    up = torch.tensor(np.repeat(rng.integers(-110, 111, C // 32), 32), dtype=torch.float64, device=G.DEV)
    x = (data(rng, M, C).double() * torch.exp2(up)).to(BF16)
    w = (data(rng, N, C).double() * torch.exp2(-up)).float()
    (xq, xs), (wq, ws) = quantised(x), quantised(w)
    y = torch.full((M, N), NAN, dtype=BF16, device=G.DEV)
    qb.qb_fp4_product(xq, xs, wq, ws, y)
    torch.cuda.synchronize()
    near4(y, xq, xs, wq, ws, C)
