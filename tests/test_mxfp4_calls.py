"""What the Python side of the MXFP4 and expert calls refuses and checks, without a GPU."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q4q():
    import __graft_entry__
    __graft_entry__.build()
    import q4_quantized_matmul_gb300 as m
    return m


def test_timeout_call_checks_its_weights(q4q):
    """Its kernel reads the whole matrix: what is not on a GPU, or too small, is refused before the launch."""
    with pytest.raises(TypeError, match="src0"):
        q4q.q4q_debug_mul_mat_mxfp4_timeout(torch.zeros(1024, dtype=torch.uint8), 64, 4, torch.zeros(1, 64), 1, 10 ** 6)


def test_experts_take_as_many_sorted_rows_as_they_give(q4q):
    """The up projection of 300000 tokens, top 4, gives 1.2 million sorted rows (fewer than 2^24): the down projection
    takes them.  Tokens, which come with slots, are limited to 2^20 as elsewhere."""
    import ctypes
    from q4_quantized_matmul_gb300 import _lib
    lib, at = _lib.load(), ctypes.c_void_p(0x1000)

    def status(n_src1, slot, rows):          # without a workspace: refused for its shape (2), or later
        return lib.q4q_mul_mat_id_mxfp4(at, 64, 32, 4, at, 0, 64, n_src1, at, slot, rows, 4, 1, at, 0, None, 0, 0, None)
    assert status(300000, at, 1200000) != 2
    assert status(1200000, None, 1200000) != 2 and status((1 << 24) - 1, None, (1 << 24) - 1) != 2
    assert status(1 << 20, at, 100) == 2 and status(1 << 24, None, 100) == 2
    n = ctypes.c_size_t(0)
    size = lib.q4q_mul_mat_id_mxfp4_workspace_size
    assert size(64, 32, 1200000, 1200000, 4, 1, ctypes.byref(n)) != 2 and size(64, 32, 1 << 24, 100, 4, 1, ctypes.byref(n)) == 2
