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


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 37, 3000])
def test_in_place(q4q, type, tokens):
    """Results over their inputs, gradients over the gradients they come from."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    q, k, gq, gk = (torch.randn(tokens, h, 96, generator=g, device="cuda").to(TYPES[type]) for h in (5, 2, 5, 2))
    qw, kw = (1 + torch.randn(96, generator=g, device="cuda") / 8 for _ in range(2))
    table, pos = q4q.q4q_rope_table(500, 48), torch.randint(0, 500, (tokens,), generator=g, device="cuda").int()
    kw_ = dict(q_weight=qw, k_weight=kw, table=table, pos=pos)
    back = q4q.q4q_qk_norm_rope_back(gq, gk, q, k, **kw_)
    got = q4q.q4q_qk_norm_rope_back(gq.clone(), gk.clone(), q, k, **kw_)
    a, b = gq.clone(), gk.clone()
    got = q4q.q4q_qk_norm_rope_back(a, b, q, k, d_q=a, d_k=b, **kw_)
    assert all(torch.equal(x, y) for x, y in zip(got, back)) and got[0].data_ptr() == a.data_ptr()
    want = q4q.q4q_qk_norm_rope(q, k, **kw_)
    got = q4q.q4q_qk_norm_rope(q, k, q_dst=q, k_dst=k, **kw_)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and got[0].data_ptr() == q.data_ptr()


@pytest.mark.parametrize("heads", [(1024, 1024), (1024, 1), (0, 1024), (1000, 0)])
@pytest.mark.parametrize("tokens", [1, 9])
def test_the_most_heads(q4q, heads, tokens):
    rng = np.random.default_rng(heads)
    q, k, gq, gk = (rng.standard_normal((tokens, h, 64)).astype(np.float32) for h in (*heads, *heads))
    w = (1 + rng.standard_normal(64) / 8).astype(np.float32)
    table, pos = ref.rope_table(50, 64), rng.integers(0, 50, tokens).astype(np.int32)
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    args = dict(q_weight=cu(w), k_weight=cu(w), table=cu(table), pos=cu(pos))
    got = q4q.q4q_qk_norm_rope(cu(q), cu(k), **args)
    for x, y in ((q, got[0]), (k, got[1])):
        assert np.array_equal(y.cpu().numpy(), ref.norm_rope(x, w, 1e-6, table, pos, True).astype(np.float32))
    dq, dk, dqw, dkw = q4q.q4q_qk_norm_rope_back(cu(gq), cu(gk), cu(q), cu(k), **args)
    for x, g, dx, dw in ((q, gq, dq, dqw), (k, gk, dk, dkw)):
        want, want_w = ref.norm_rope_back(g, x, w, 1e-6, table, pos, True)
        # results of the size of 1, sums of up to 9 2^10 terms of it
        assert np.all(np.abs(dx.cpu().numpy() - want) <= 2.0 ** -17 * (1 + np.abs(want)))
        assert np.all(np.abs(dw.cpu().numpy() - want_w) <= 2.0 ** -24 * (tokens * x.shape[1] / 8 + 64) * np.abs(g).sum((0, 1)) * 8)
    if heads[1]:
        cache = torch.zeros(2 * q4q.q4q_kv_page_size(heads[1], 64, 16), dtype=torch.uint8, device="cuda")
        slots = rng.permutation(32)[:tokens].astype(np.int32)
        q4q.q4q_kv_append(cache, 16, cu(k), cu(gk), cu(slots))
        assert np.array_equal(cache.cpu().numpy(), ref.put(np.zeros(cache.numel(), np.uint8), 16, slots, k, gk))
        a, b = q4q.q4q_kv_get_rows(cache, 16, heads[1], 64, cu(slots))
        want = ref.get(cache.cpu().numpy(), 16, heads[1], 64, slots)
        assert np.array_equal(a.double().cpu().numpy(), want[0]) and np.array_equal(b.double().cpu().numpy(), want[1])
    assert q4q.q4q_device_status() == 0


def test_rows_past_2_to_the_32(q4q):
    """Tokens 2^30 elements apart, as the views of a buffer of 10 GB: the same as of one without gaps."""
    buf = torch.empty(4 * 2 ** 30 + 8 * 64 * 4, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(5, 8, 64, device="cuda").bfloat16()
    far = buf.as_strided((5, 8, 64), (2 ** 30, 64, 1))
    far.copy_(x)
    w, table, pos = torch.ones(64, device="cuda"), q4q.q4q_rope_table(8, 64), torch.arange(5, dtype=torch.int32, device="cuda")
    args = dict(q_weight=w, k_weight=w, table=table, pos=pos)
    for a, b in zip(q4q.q4q_qk_norm_rope(far, far, **args), q4q.q4q_qk_norm_rope(x, x, **args)):
        assert torch.equal(a, b)
    for a, b in zip(q4q.q4q_qk_norm_rope_back(x, x, far, far, **args), q4q.q4q_qk_norm_rope_back(x, x, x, x, **args)):
        assert torch.equal(a, b)
    one, two = (torch.zeros(q4q.q4q_kv_page_size(8, 64, 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    assert torch.equal(q4q.q4q_kv_append(one, 16, far, far, pos, w, 1e-6, table, pos), q4q.q4q_kv_append(two, 16, x, x, pos, w, 1e-6, table, pos))
    pages, length, first = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[0]], [5], [0, 5]))
    assert torch.equal(q4q.q4q_kv_attn(far, one, 16, 8, pages, length, first=first), q4q.q4q_kv_attn(x, one, 16, 8, pages, length, first=first))
    assert q4q.q4q_device_status() == 0
