"""The exchange at the ends of the sizes that its calls accept."""
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


def test_the_most_pairs_of_one_expert():
    """2^31 - 2 pairs of one expert, a multiple of 3, rounded up to one: the
    rows stay below 2^31, pairs + align - 1 does not."""
    N, K, E, align = (1 << 30) - 1, 2, 1, 3
    R = qb.qb_dispatch_rows(N, K, E, align)
    assert R == N * K == (1 << 31) - 2
    i32 = dict(dtype=torch.int32, device=G.DEV)
    G.say(f"dispatch of {N * K} pairs")
    topk = torch.zeros((N, K), **i32)
    off, src, pos = torch.full((E + 1,), -7, **i32), torch.full((R,), -7, **i32), torch.full((N, K), -7, **i32)
    ws = torch.empty(qb.qb_dispatch_workspace_bytes(N, K, E), dtype=torch.uint8, device=G.DEV)
    qb.qb_dispatch(topk, E, align, off, src, pos, ws)
    torch.cuda.synchronize()
    assert off.tolist() == [0, R]
    flat, step = pos.view(-1), 1 << 28
    for a in range(0, R, step):
        n = min(step, R - a)
        i = torch.arange(a, a + n, **i32)
        assert torch.equal(flat[a:a + n], i) and torch.equal(src[a:a + n], i // K)
    del topk, src, pos, flat, i
    torch.cuda.empty_cache()
