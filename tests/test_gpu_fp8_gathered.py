"""Quantising rows taken by number (row_src) from inputs that pass the caches
by and from inputs that are kept in them: the same bytes as from the rows laid
out one after the other."""
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


def quantised(x, M, C, src=None):
    q = torch.full((M, qb.fp8_ld(C)), 0x55, dtype=torch.uint8, device=G.DEV).view(qb.F8)
    s = torch.full((M, qb.fp8_sld(C)), 0x55, dtype=torch.uint8, device=G.DEV)
    qt = torch.full((C, qb.fp8_ld(M)), 0x55, dtype=torch.uint8, device=G.DEV).view(qb.F8)
    st = torch.full((C, qb.fp8_sld(M)), 0x55, dtype=torch.uint8, device=G.DEV)
    qb.qb_fp8_quantize(x, q, s, row_src=src)
    qb.qb_fp8_quantize_cols(x, qt, st, row_src=src)
    torch.cuda.synchronize()
    return q.view(torch.uint8), s, qt.view(torch.uint8), st


# 128 MiB and more, each row once and more than twice; a small input for many rows
@pytest.mark.parametrize("Mx,M,C", [(70001, 70100, 1000), (70001, 150003, 1000), (1001, 70003, 1030)])
def test_rows_by_number_of_large_inputs(Mx, M, C):
    g = torch.Generator(device=G.DEV).manual_seed(M)
    x = torch.randn((Mx, C), generator=g, device=G.DEV).to(torch.bfloat16)
    src = torch.randint(-1, Mx, (M,), generator=g, device=G.DEV, dtype=torch.int32)
    G.say(f"quantise by row number Mx={Mx} M={M} C={C}")
    laid = torch.where((src >= 0)[:, None], x[src.clamp(min=0).long()], torch.zeros((), dtype=x.dtype, device=G.DEV))
    for name, got, ref in zip(("q", "scales", "transposed", "its scales"), quantised(x, M, C, src), quantised(laid, M, C)):
        n = -(-(C if name == "scales" else M) // 128) if "scales" in name else got.shape[1]
        assert torch.equal(got[:, :n], ref[:, :n]), name
