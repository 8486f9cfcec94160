"""The experts' products write nothing but their results and workspace, whatever stands in `first`.

Kernels clamp what they read from `first` to the rows that there are, and a segment to the tiles that the
workspace holds, so wrong entries give wrong rows and no access out of bounds.  Results and workspace lie
inside larger buffers here, whose other bytes have to stay as they were.
"""
import numpy as np
import pytest

from mx_forms import sizes
from test_gpu_mxfp4 import q4q  # noqa: F401
from test_gpu_mxfp4_forms import lib_and_sms, operands

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EDGE, MARK = 1 << 20, 0xA5          # bytes on either side, and what they hold


class Inside:
    """`count` bytes in the middle of a marked buffer."""

    def __init__(self, count):
        self.buffer = torch.full((count + 2 * EDGE,), MARK, dtype=torch.uint8, device="cuda")
        self.bytes = self.buffer[EDGE:EDGE + count]

    def untouched(self):
        return bool((self.buffer[:EDGE] == MARK).all()) and bool((self.buffer[EDGE + self.bytes.numel():] == MARK).all())


def wrong_firsts(rng, experts, n):
    """Out of range, falling, jumping up and down, and random."""
    top = 2 ** 31 - 1
    yield [0] + [top] * experts
    yield [top] * (experts + 1)
    yield [-5] * (experts + 1)
    yield [n - i * (n // max(experts, 1)) for i in range(experts + 1)]
    yield [n if i % 2 else 0 for i in range(experts + 1)]
    yield [0 if i % 2 else n + 3 for i in range(experts + 1)]
    for _ in range(3):
        yield rng.integers(-n, 2 * n, experts + 1).tolist()


@pytest.mark.parametrize("acts", [0, 1])
@pytest.mark.parametrize("wanted", [(8, 1, 1), (8, 1, 8), (16, 1, 4), (32, 1, 2), (64, 1, 1), (64, 1, 8), (64, 2, 1), (128, 2, 1), (256, 2, 1)],
                         ids=lambda f: "%d-%d-%d" % f)
def test_wrong_firsts_stay_in_bounds(q4q, wanted, acts):  # noqa: F811
    lib, sms = lib_and_sms()
    k, rows, tokens, top, experts = sizes(lib, acts, True, sms)[wanted]
    n = tokens * top
    g = torch.Generator(device="cuda").manual_seed(7)
    packed, _, x = operands(q4q, g, k, rows, tokens, experts, acts)
    slot = torch.randperm(n, generator=g, device="cuda").int()
    dst, ws = Inside(n * rows * 4), Inside(q4q.q4q_mul_mat_id_mxfp4_workspace_size(k, rows, tokens, n, experts, acts))
    y = dst.bytes.view(torch.float32).view(n, rows)

    def product(first, out, work):
        return q4q.q4q_mul_mat_id_mxfp4(packed, k, rows, x, torch.tensor(first, dtype=torch.int32, device="cuda"), slot, top, acts, dst=out, workspace=work)
    for first in wrong_firsts(np.random.default_rng([k, n]), experts, n):
        product(first, y, ws.bytes)
        assert dst.untouched() and ws.untouched(), first
        assert q4q.q4q_device_status() == 0
    # ends past the last row are the last row
    ends = sorted(np.random.default_rng(n).integers(0, n, experts - 1).tolist())
    product([0] + ends + [n], y, ws.bytes)
    right = y.clone()
    product([-9] + ends + [n + 1000], y, ws.bytes)
    assert torch.equal(y, right) and dst.untouched() and ws.untouched()
