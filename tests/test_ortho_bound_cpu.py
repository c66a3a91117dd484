"""The bound on qb_orthogonalize's results refuses the update with a part or a
pass left out: planted in the simulation, on the CPU."""
import pytest
import torch

from ortho_forms import above_rounding, bound, formula, held

LEFT_OUT = [("x",), ("S",), ("P",), ("add x",), ("add S",), ("S: hl", "S: lh"), ("S: hl",), ("SS: hl", "SS: lh"), ("SS: lh",), ("Px: hl",),
            ("Px: lh",), ("Px: hl", "Px: lh")]


def matrix(N, C):
    return torch.randn((N, C), generator=torch.Generator().manual_seed(N + C))


@pytest.mark.parametrize("N,C", [(1, 1), (1, 300), (16, 16), (33, 70), (128, 256), (301, 165), (512, 640)])
def test_the_whole_form_keeps_it(N, C):
    x = matrix(N, C)
    want = formula(x)
    assert above_rounding(held(x).to(torch.bfloat16), want) <= bound(x, want)


@pytest.mark.parametrize("without", LEFT_OUT, ids=" ".join)
@pytest.mark.parametrize("N,C", [(128, 256), (301, 165), (512, 640)])
def test_a_form_without_a_part_exceeds_it(N, C, without):
    x = matrix(N, C)
    want = formula(x)
    assert above_rounding(held(x, without=without).to(torch.bfloat16), want) > bound(x, want)
