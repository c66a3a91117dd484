"""The expert layer's calls as a program makes them, on the host alone."""
import inspect


def test_a_product_holds_its_sums_in_32_bits_unless_the_caller_says_otherwise():
    from exact_quantile_selection_amd import qb
    from exact_quantile_selection_amd.expert_layer import ExpertLayer

    assert inspect.signature(qb.qb_fp8_product).parameters["exact"].default is True
    assert inspect.signature(ExpertLayer).parameters["exact"].default is True
