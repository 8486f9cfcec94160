"""The choice among the forms of the MXFP4 products, on the host alone."""
import ctypes

import pytest

from mx_forms import FORMS, form, sizes


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from q4_quantized_matmul_gb300 import _lib
    return _lib.load()


@pytest.mark.parametrize("acts", [0, 1])
@pytest.mark.parametrize("by_expert", [False, True])
@pytest.mark.parametrize("sms", [152, 148, 132])
def test_every_form_is_within_reach_of_the_tests(lib, sms, by_expert, acts):
    assert set(sizes(lib, acts, by_expert, sms)) == set(FORMS)


def test_form_of_known_sizes(lib):
    """As launched on a GB300 (152 SMs)."""
    for (k, rows, tokens, acts), want in {(4096, 14336, 1, 1): (8, 1, 1), (14336, 4096, 33, 1): (64, 1, 4), (4096, 14336, 512, 1): (256, 2, 1),
                                          (14336, 4096, 2048, 0): (256, 2, 1)}.items():
        assert form(lib, k, rows, tokens, tokens, 0, acts, 152) == want
    assert form(lib, 1504, 777, 517 * 4, 517, 32, 1, 152) == (128, 2, 1)


def test_refusals_of_the_form_query(lib):
    out = (ctypes.c_int * 3)()
    f = lib.q4q_debug_mxfp4_form
    assert f(64, 4, 1, 1, 0, 1, 152, None) == 1
    assert f(33, 4, 1, 1, 0, 1, 152, out) == 2 and f(64, 0, 1, 1, 0, 1, 152, out) == 2
    assert f(64, 4, 0, 1, 0, 1, 152, out) == 2 and f(64, 4, 1, 1 << 24, 0, 1, 152, out) == 2
    assert f(64, 4, 1, 1, -1, 1, 152, out) == 7 and f(64, 4, 1, 1, 1025, 1, 152, out) == 7
    assert f(64, 4, 1, 1, 0, 2, 152, out) == 7 and f(64, 4, 1, 1, 0, 1, 1, out) == 7
