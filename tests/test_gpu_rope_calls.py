"""Calls of norm and rotation and of the cache that their documentation allows and that take little."""
import pytest

from test_gpu_rope_kv import q4q  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_a_table_without_positions(q4q):
    """Is refused (rows came back as if there were no table), but for a call without tokens."""
    x, pos = torch.randn(4, 3, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    cache = torch.full((q4q.q4q_kv_page_size(3, 64, 16),), 7, dtype=torch.uint8, device="cuda")
    for table in (torch.empty(0, 64, device="cuda"), torch.empty(8, 0, device="cuda")):
        for call in (lambda: q4q.q4q_qk_norm_rope(x, x, table=table, pos=pos), lambda: q4q.q4q_qk_norm_rope_back(x, None, x, table=table, pos=pos),
                     lambda: q4q.q4q_kv_append(cache, 16, x, x, pos, table=table, pos=pos)):
            with pytest.raises(ValueError):
                call()
    assert (cache == 7).all()
    assert q4q.q4q_qk_norm_rope(x[:0], table=torch.empty(0, 64, device="cuda"), pos=pos)[0].shape == (0, 3, 64)
    assert q4q.q4q_device_status() == 0
