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


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_at_the_limits_of_their_range(q4q, dim, eps):
    """Forward to the bit, backward within the bound of test_gpu_rope_kv's gradients: roundings of sums and products, in units of each row's
    result."""
    rng = np.random.default_rng(dim)
    x = rng.standard_normal((9, 2, dim)).astype(np.float32)
    x /= np.sqrt((x.astype(np.float64) ** 2).mean(-1, keepdims=True)).astype(np.float32)
    for i, size in enumerate((2.0 ** -44.9, 2.0 ** -40, 2.0 ** -20, 1.0, 2.0 ** 20, 2.0 ** 40, 2.0 ** 57)):
        x[i] *= np.float32(size)
    x[7:] = np.nextafter(np.float32(2.0 ** 60), np.float32(0)) * np.sign(x[7:])
    w, g = (1 + 0.3 * rng.standard_normal(dim)).astype(np.float32), rng.standard_normal(x.shape).astype(np.float32)
    cx, cw, cg = (torch.from_numpy(a).cuda() for a in (x, w, g))
    got, _ = q4q.q4q_qk_norm_rope(cx, q_weight=cw, eps=eps)
    got, want = got.cpu().numpy(), ref.norm_rope(x, w, eps, None, None, True).astype(np.float32)
    assert np.array_equal(got[:7], want[:7])
    # The last rows' values are all 2^60 (1 - 2^-24) in size, so r = 2^-60 (1 + 2^-24 + 2^-48 + ...) is 2^-48 of itself past the middle of two
    # fp32, nearer than sums and products in two fp32 (2^-47) tell: either of the two, 2^-23 apart, is right, and x r and (x r) w round once more each.
    assert np.all(np.abs(got[7:].astype(np.float64) - want[7:]) <= np.abs(want[7:]) * (2.0 ** -23 + 2 * 2.0 ** -24))
    dx, _, dw, _ = q4q.q4q_qk_norm_rope_back(cg, None, cx, None, cw, None, eps)
    want, want_w = ref.norm_rope_back(g, x, w, eps, None, None, True)
    x64 = x.astype(np.float64)
    r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + float(np.float32(eps)))
    dh, xh, u = np.abs(g * w), np.abs(x64 * r), 2.0 ** -24
    assert np.all(np.abs(dx.double().cpu().numpy() - want) <= (dim / 8 + 24) * u * r * (dh + xh * (dh * xh).mean(-1, keepdims=True)) + 2.0 ** -149)
    assert np.all(np.abs(dw.double().cpu().numpy() - want_w) <= (18 + 64) * u * (np.abs(g) * xh).sum((0, 1)))


def test_many_rows_of_large_values(q4q):
    """Up to 2^60: as exact as rows of ordinary values."""
    rng = np.random.default_rng(60)
    x = (rng.uniform(-1, 1, (6000, 1, 64)) * 2.0 ** 60).astype(np.float32)
    w = np.ones(64, np.float32)
    got, _ = q4q.q4q_qk_norm_rope(torch.from_numpy(x).cuda(), q_weight=torch.from_numpy(w).cuda(), eps=0.0)
    assert np.array_equal(got.cpu().numpy(), ref.norm_rope(x, w, 0.0, None, None, True).astype(np.float32))
