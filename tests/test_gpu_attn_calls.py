"""Attention over the cache: workspaces, and cases that take much memory."""
import numpy as np
import pytest

from oracle import attn as ref
from test_gpu_attn import Case, TYPES, check, on_tensor_cores, q4q, widened  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_one_workspace_for_all_batches(q4q, type, dim):
    """A size asked for the most rows and sequences serves fewer of either."""
    most = q4q.q4q_kv_attn_workspace_size(300, 4, 2, dim, 300, TYPES[type])
    for n_q in (1, 31, 32, 33, 150, 300):
        for n_seqs in (1, 2, 5, 150, 300):
            assert q4q.q4q_kv_attn_workspace_size(n_q, 4, 2, dim, n_seqs, TYPES[type]) <= most
    ws = torch.zeros(most, dtype=torch.uint8, device="cuda")
    for lengths, rows in (([40] * 150, [2] * 150), ([400], [300]), ([300, 90], [140, 60])):
        case = Case([dim, len(rows)], lengths, rows, 4, 2, dim, 16, type)
        got = case.run(q4q, workspace=ws)
        check(case, got)
        case = widened(case)
        check(case, case.run(q4q, workspace=ws))
