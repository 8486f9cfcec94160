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
