"""Arguments, errors and limits of the MXFP4 and expert calls on the GPU."""
import numpy as np
import pytest

from oracle import mx
from test_gpu_mxfp4 import close, on_gpu, q4q, rand  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_timeout_call_checks_its_weights(q4q):  # noqa: F811
    """A matrix that is too small is refused before the launch."""
    x = torch.zeros(1, 64, device="cuda")
    small = torch.zeros(q4q.q4q_mxfp4_size(64, 200) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="src0"):
        q4q.q4q_debug_mul_mat_mxfp4_timeout(small, 64, 200, x, 1, 10 ** 6)
    with pytest.raises(TypeError, match="src0"):
        q4q.q4q_debug_mul_mat_mxfp4_timeout(small.cpu(), 64, 200, x, 1, 10 ** 6)
    assert q4q.q4q_device_status() == 0


def test_memory_that_is_not_there_is_torchs_error(q4q):  # noqa: F811
    """A million rows of half a million values do not fit: the error is the one that a program catches from torch."""
    tokens, top = 1000, 1000
    first, slot, row = q4q.q4q_moe_sort(torch.zeros(tokens, top, dtype=torch.int32, device="cuda"), 4)
    src = torch.zeros(tokens, 1 << 19, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        q4q.q4q_moe_gather(src, first, row, top)
    assert q4q.q4q_moe_gather(src[:, :8].contiguous(), first, row, top).shape == (tokens * top, 8)


def test_refused_calls_take_no_memory(q4q):  # noqa: F811
    """A mistyped size is refused before results of that size are allocated (gigabytes, in these calls)."""
    u8 = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    x, ids = torch.zeros(3, 64, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    first, slot, row = q4q.q4q_moe_sort(ids, 4)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for error, call in (
            (q4q.Q4QError, lambda: q4q.q4q_moe_sort(ids, 2 ** 30)),
            (q4q.Q4QError, lambda: q4q.q4q_moe_sort(ids, 0)),
            (ValueError, lambda: q4q.q4q_moe_gather(x, first, row, 2 ** 20)),
            (ValueError, lambda: q4q.q4q_get_rows_mxfp4(u8, 64, 2 ** 24)),
            (ValueError, lambda: q4q.q4q_mul_mat_mxfp4(u8, 64, 2 ** 28, x)),
            (ValueError, lambda: q4q.q4q_mul_mat_id_mxfp4(u8, 64, 2 ** 28, x, first, slot, 2))):
        with pytest.raises(error):
            call()
    assert torch.cuda.max_memory_allocated() == before


def test_a_million_sorted_rows(q4q):  # noqa: F811
    """1,100,000 rows that are sorted already, more than there may be tokens; three experts, K = 32."""
    n, rows, experts = 1100000, 24, 3
    rng = np.random.default_rng(41)
    packs = [mx.pack(rand(rng, rows, 32, 0.05).astype(np.float32)) for _ in range(experts)]
    w = torch.from_numpy(np.stack([p[0] for p in packs])).cuda()
    x, v = on_gpu(rand(rng, n, 32), "bf16")
    at = [0, 5, 600001, n - 1000]                              # the last 1000 rows are nobody's
    first = torch.tensor(at, dtype=torch.int32, device="cuda")
    got = q4q.q4q_mul_mat_id_mxfp4(w, 32, rows, x, first, dst_dtype=torch.float32)
    assert not got[at[3]:].any()
    for e in range(experts):
        for r in (slice(at[e], min(at[e] + 300, at[e + 1])), slice(max(at[e + 1] - 300, at[e]), at[e + 1])):
            a = mx.encode(v[r], "mxfp8")[2]
            close(got[r], a @ packs[e][1].T, np.abs(a) @ np.abs(packs[e][1]).T, 32, "f32")
    assert q4q.q4q_device_status() == 0
