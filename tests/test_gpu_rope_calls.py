"""Calls of norm and rotation and of the cache that their documentation allows and that take little."""
import numpy as np
import pytest

from oracle import attn as ref
from test_gpu_rope_kv import TYPES, q4q  # noqa: F401

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


@pytest.mark.parametrize("type", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads", [(64, 1), (96, 1), (96, 5), (128, 3), (256, 2)])
def test_append_of_16_bit_rows_with_zero_blocks(q4q, type, dim, heads):
    """Quotients on half steps beside blocks of zeros, of subnormal numbers and lanes without values, in one warp."""
    rng = np.random.default_rng([dim, heads])
    k, v = (torch.from_numpy((rng.integers(-16, 17, (40, heads, dim)) / 8).astype(np.float32)).to(TYPES[type]) for _ in range(2))
    zero = torch.from_numpy(rng.integers(0, 3, (40, heads, dim // 32)).repeat(32, 2))
    k[zero == 0], v[zero == 1] = 0, 0
    v[7] *= 2.0 ** -14 if type == "f16" else 2.0 ** -130
    slots = rng.permutation(64)[:40].astype(np.int32)
    cache = torch.zeros(4 * q4q.q4q_kv_page_size(heads, dim, 16), dtype=torch.uint8, device="cuda")
    q4q.q4q_kv_append(cache, 16, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    want = ref.put(np.zeros(cache.numel(), np.uint8), 16, slots, k.float().numpy(), v.float().numpy())
    assert np.array_equal(cache.cpu().numpy(), want)
