"""The MXFP4 and expert entry points without a GPU: refusals, sizes, and the plain reference's own pins."""
import ctypes

import numpy as np
import pytest

from oracle import mx

P = ctypes.c_void_p
FAKE, ODD = P(0x1000), P(0x1002)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from q4_quantized_matmul_gb300 import _lib
    return _lib.load()


def test_sizes(lib):
    n = ctypes.c_size_t(0)
    for k, rows in [(32, 1), (256, 128), (288, 129), (4096, 777)]:
        assert lib.q4q_mxfp4_size(k, rows, ctypes.byref(n)) == 0
        assert n.value == mx.pack(np.zeros((rows, k), np.float32))[0].size and n.value % 256 == 0
    assert lib.q4q_mxfp4_size(33, 4, ctypes.byref(n)) == 2
    assert lib.q4q_mxfp4_size(32, -1, ctypes.byref(n)) == 2
    assert lib.q4q_mxfp4_size(32, 4, None) == 1


def test_refusals_of_encoder_and_rows(lib):
    f = lib.q4q_quantize_mxfp4
    assert f(FAKE, 0, FAKE, 31, 2, 1, None) == 2
    assert f(FAKE, 0, FAKE, 32, -1, 1, None) == 2
    assert f(FAKE, 0, FAKE, 32, 2, -1, None) == 2
    assert f(FAKE, 0, FAKE, 1 << 19, 1 << 20, 4, None) == 2                       # too many elements
    assert f(FAKE, 3, FAKE, 32, 2, 1, None) == 7
    assert f(None, 0, FAKE, 32, 2, 1, None) == 1
    assert f(ODD, 0, FAKE, 32, 2, 1, None) == 3
    assert f(FAKE, 0, P(0x1080), 32, 2, 1, None) == 3                             # dst not 256-byte aligned
    assert f(None, 0, None, 32, 0, 1, None) == 0
    assert f(None, 0, None, 32, 2, 0, None) == 0
    g = lib.q4q_get_rows_mxfp4
    assert g(FAKE, 48, 10, FAKE, 3, FAKE, None) == 2
    assert g(FAKE, 64, 10, None, 11, FAKE, None) == 2
    assert g(FAKE, 64, 10, FAKE, -1, FAKE, None) == 2
    assert g(FAKE, 64, 10, FAKE, 0, FAKE, None) == 0
    assert g(None, 64, 10, FAKE, 3, FAKE, None) == 1
    assert g(P(0x1010), 64, 10, FAKE, 3, FAKE, None) == 3
    assert g(FAKE, 64, 10, FAKE, 3, P(0x1004), None) == 3
    assert g(FAKE, 64, 10, ODD, 3, FAKE, None) == 3


def test_refusals_of_the_product(lib):
    def f(src0=FAKE, ne00=64, ne01=4, src1=FAKE, t1=0, ne10=64, ne11=2, acts=1, dst=FAKE, t2=0, flags=0):
        return lib.q4q_mul_mat_mxfp4(src0, ne00, ne01, src1, t1, ne10, ne11, acts, dst, t2, None, 0, flags, None)
    assert f(ne00=33, ne10=33) == 2
    assert f(ne10=96) == 2
    assert f(ne01=-1) == 2 and f(ne11=-1) == 2 and f(ne11=1 << 20) == 2
    assert f(t1=3) == 7 and f(t2=-1) == 7 and f(acts=2) == 7 and f(flags=2) == 7
    assert f(src0=None) == 1 and f(src1=None) == 1 and f(dst=None) == 1
    assert f(src0=P(0x1010)) == 3 and f(src1=ODD) == 3 and f(dst=ODD) == 3
    assert f(src0=None, ne01=0) == 0 and f(src1=None, ne11=0) == 0
    n = ctypes.c_size_t(0)
    w = lib.q4q_mul_mat_mxfp4_workspace_size
    assert w(48, 4, 1, 1, ctypes.byref(n)) == 2 and w(64, 4, 1, 2, ctypes.byref(n)) == 7 and w(64, 4, 1, 1, None) == 1
    assert w(64, 0, 1, 1, ctypes.byref(n)) == 0 and n.value == 0
    d = lib.q4q_debug_mul_mat_mxfp4_timeout
    assert d(FAKE, 64, 4, FAKE, 1, 1, FAKE, None, 0, 0, None) == 7
    assert d(FAKE, 64, 4, FAKE, 1, 1, FAKE, None, 0, 2 * 10 ** 9, None) == 7
    assert d(FAKE, 64, 0, FAKE, 1, 1, FAKE, None, 0, 10 ** 6, None) == 2


def test_refusals_of_the_experts(lib):
    s = lib.q4q_moe_sort
    assert s(FAKE, -1, 2, 4, FAKE, FAKE, FAKE, None) == 2
    assert s(FAKE, 1 << 30, 2, 4, FAKE, FAKE, FAKE, None) == 2
    assert s(FAKE, 3, 0, 4, FAKE, FAKE, FAKE, None) == 7
    assert s(FAKE, 3, 2, 0, FAKE, FAKE, FAKE, None) == 7
    assert s(FAKE, 3, 2, 1025, FAKE, FAKE, FAKE, None) == 7
    assert s(None, 3, 2, 4, FAKE, FAKE, FAKE, None) == 1 and s(FAKE, 3, 2, 4, None, FAKE, FAKE, None) == 1
    assert s(ODD, 3, 2, 4, FAKE, FAKE, FAKE, None) == 3
    for g in (lib.q4q_moe_gather, lib.q4q_moe_gather_back):
        assert g(FAKE, 0, 0, 3, 2, FAKE, 4, FAKE, FAKE, None) == 2
        assert g(FAKE, 9, 8, 3, 2, FAKE, 4, FAKE, FAKE, None) == 7
        assert g(FAKE, 0, 8, 3, 0, FAKE, 4, FAKE, FAKE, None) == 7
        assert g(None, 0, 8, 3, 2, FAKE, 4, FAKE, FAKE, None) == 1
        assert g(FAKE, 0, 8, 3, 2, FAKE, 4, ODD, FAKE, None) == 3
        assert g(None, 0, 8, 0, 2, None, 4, None, None, None) == 0
    c = lib.q4q_moe_combine
    assert c(FAKE, 0, 8, 3, 2, FAKE, 4, FAKE, None, FAKE, None) == 1
    assert c(FAKE, 0, 8, 3, 2, FAKE, 4, FAKE, ODD, FAKE, None) == 3
    assert c(FAKE, 0, 8, 0, 2, FAKE, 4, FAKE, None, FAKE, None) == 0
    b = lib.q4q_moe_combine_back
    assert b(FAKE, FAKE, 0, 8, 3, 2, FAKE, 4, FAKE, FAKE, FAKE, None, None) == 1
    assert b(FAKE, ODD, 0, 8, 3, 2, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None) == 3

    def f(src0=FAKE, ne00=64, ne01=4, e=4, src1=FAKE, ne10=64, n1=3, first=FAKE, slot=FAKE, rows=6, k=2, acts=1, dst=FAKE):
        return lib.q4q_mul_mat_id_mxfp4(src0, ne00, ne01, e, src1, 0, ne10, n1, first, slot, rows, k, acts, dst, 0, None, 0, 0, None)
    assert f(ne00=33, ne10=33) == 2 and f(ne10=32) == 2
    assert f(e=0) == 7 and f(e=1025) == 7 and f(k=0) == 7 and f(acts=7) == 7
    assert f(rows=7) == 2 and f(rows=4, slot=None) == 2 and f(rows=-1) == 2
    assert f(first=None) == 1 and f(src0=None) == 1 and f(dst=None) == 1
    assert f(src0=P(0x1010)) == 3 and f(slot=ODD) == 3
    assert f(rows=0) == 0 and f(ne01=0) == 0


def test_bindings_refuse_what_they_cannot_take():
    import torch
    import q4_quantized_matmul_gb300 as q4q
    with pytest.raises(TypeError):
        q4q.q4q_quantize_mxfp4(torch.zeros(2, 32))                                # not on a GPU
    with pytest.raises(TypeError):
        q4q.q4q_quantize_mxfp4(torch.zeros(2, 32, dtype=torch.float64))
    with pytest.raises(TypeError):
        q4q.q4q_moe_sort(torch.zeros(2, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        q4q.q4q_moe_sort(torch.zeros(2, dtype=torch.int32), 4)


def test_reference_rounds_as_the_format_says():
    # E2M1 ties go to the even code, values above 6 to 6
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    assert list(mx.E2M1[mx.nearest(v, mx.E2M1)]) == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    assert mx.E4M3[-1] == 448.0 and mx.E4M3[1] == 2.0 ** -9 and mx.E4M3[8] == 2.0 ** -6
    x = np.zeros((1, 64), np.float32)
    x[0, 0], x[0, 1], x[0, 40] = 7.0, -0.4, np.inf
    codes, scales, values = mx.encode(x, "mxfp4")
    assert scales.tolist() == [[127, 255]] and codes[0, 0] == 7 and codes[0, 1] == 9 and np.isnan(values[0, 32:]).all()
    assert mx.encode(np.zeros((1, 32), np.float32), "mxfp4")[1].tolist() == [[0]]


def test_reference_layout_of_a_matrix():
    w = np.zeros((130, 288), np.float32)
    w[129, 257] = -3.0                                     # block 8: second 128-row group, third column chunk
    packed, values = mx.pack(w)
    codes = mx.up(130 * 256, 256)
    assert packed[129 * 256 + 128] == (0xF << 4)           # scale 2^-1, so minus the code of 6; odd element: high nibble
    assert packed[codes + (1 * 4 + 2) * 512 + 1 * 16 + 0 * 4 + 0] == 126
    assert values[129, 257] == -3.0 and np.count_nonzero(packed) == 2


def test_reference_sort_keeps_slot_order():
    first, slot, row = mx.sort(np.array([[1, -1], [0, 1], [5, 0]]), 3)
    assert first.tolist() == [0, 2, 4, 4] and slot.tolist() == [2, 5, 0, 3, 1, 4] and row.tolist() == [2, 4, 0, 3, 5, 1]
