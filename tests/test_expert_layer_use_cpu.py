"""The expert layer's calls as a program makes them, on the host alone."""
import inspect
import os

import pytest

FAKE = 0x1000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    from exact_quantile_selection_amd import build, qb

    if not os.path.exists(qb.LIB_PATH):
        build.build()
    return qb.lib()


def test_a_product_holds_its_sums_in_32_bits_unless_the_caller_says_otherwise():
    from exact_quantile_selection_amd import qb
    from exact_quantile_selection_amd.expert_layer import ExpertLayer

    assert inspect.signature(qb.qb_fp8_product).parameters["exact"].default is True
    assert inspect.signature(ExpertLayer).parameters["exact"].default is True


def test_the_refusals_of_what_leaves_rows_out(L):
    import torch

    from exact_quantile_selection_amd import qb

    def refused(status, words, rc):
        assert rc == getattr(qb, status), (rc, L.qb_last_error())
        assert words in L.qb_last_error().decode()

    clear = lambda s=FAKE, topk=FAKE, n=10, e=16, k=2: L.qb_unrouted_clear(s, topk, n, e, k, None)  # noqa: E731
    count = lambda topk=FAKE, n=10, e=16, k=2, a=FAKE, h=FAKE: (  # noqa: E731
        L.qb_unrouted_uncount(topk, n, e, k, a, h, None))
    for call in (clear, count):
        refused("QB_EINVAL", "N=0", call(n=0))
        refused("QB_EINVAL", "2^31", call(n=1 << 31))
        refused("QB_EUNSUPPORTED", "E=48", call(e=48))
        refused("QB_EINVAL", "K=16", call(k=16))
        refused("QB_EINVAL", "K=0", call(k=0))
        refused("QB_EINVAL", "topk is NULL", call(topk=None))
        refused("QB_EINVAL", "4-byte", call(topk=FAKE + 2))
    refused("QB_EINVAL", "s is NULL", clear(s=None))
    refused("QB_EINVAL", "16-byte", clear(s=FAKE + 4))
    refused("QB_EINVAL", "required", count(a=None))
    refused("QB_EINVAL", "required", count(h=None))
    refused("QB_EINVAL", "8-byte", count(h=FAKE + 4))
    refused("QB_EINVAL", "4-byte", count(a=FAKE + 1))
    s, ids = torch.zeros((4, 16)), torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="s must be a GPU tensor"):
        qb.qb_unrouted_clear(s, ids)
    with pytest.raises(ValueError, match="topk must be a GPU tensor"):
        qb.qb_unrouted_uncount(ids, s[0], torch.zeros((16, 256), dtype=torch.int32))
    with pytest.raises(ValueError, match="must be"):
        qb.qb_unrouted_clear(s[0], ids)
