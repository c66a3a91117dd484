"""Who chooses how many bits the orthogonalised update takes, and what its coarse
form refuses, on the host alone."""
import inspect
import os

import pytest

FAKE = 0x1000  # never dereferenced: validation fails first


def test_fewer_bits_are_the_callers_choice():
    from exact_quantile_selection_amd import qb
    from exact_quantile_selection_amd.expert_layer import ExpertLayer

    assert inspect.signature(qb.qb_orthogonalize).parameters["exact"].default is True
    assert inspect.signature(ExpertLayer.orthogonalized).parameters["exact"].default is True


def test_the_coarse_form_refuses_what_the_other_does():
    from exact_quantile_selection_amd import build, qb

    if not os.path.exists(qb.LIB_PATH):
        build.build()
    L = qb.lib()
    need = L.qb_orthogonalize_workspace_bytes(2, 10, 20)
    o = lambda x=FAKE, g=2, n=10, c=20, steps=5, out=FAKE, ws=FAKE, b=need: (  # noqa: E731
        L.qb_orthogonalize_coarse(x, g, n, c, steps, 1.5, -0.5, 0.0, out, ws, b, None))
    for words, kw in (("G=0", dict(g=0)), ("N=0", dict(n=0)), ("C=65537", dict(c=65537)), ("steps=65", dict(steps=65)),
                      ("required", dict(x=None)), ("required", dict(out=None)), ("ws_bytes=0", dict(ws=None)),
                      ("qb_orthogonalize_workspace_bytes", dict(b=need - 1)), ("16-byte", dict(ws=FAKE + 8)),
                      ("2-byte", dict(out=FAKE + 1)), ("4-byte", dict(x=FAKE + 2))):
        assert o(**kw) == qb.QB_EINVAL
        said = L.qb_last_error().decode()
        assert words in said and said.startswith("qb_orthogonalize_coarse"), said


def test_the_coarse_form_names_a_wrong_tensor():
    import torch

    from exact_quantile_selection_amd import qb

    x = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        qb.qb_orthogonalize(x, x, x, exact=False)
