"""Norms and rotation of queries and keys, their gradients, and the cache's append and row gather, against oracle/attn.py.

Norm, rotation and encoding are defined to the last bit (each product, difference and sum rounded to fp32, the norm's
factor that of 64-bit sums), so results and cache bytes are compared for equality.  The norm's factor is computed in
pairs of fp32 to about 2^-45, so one row in 2^20 may get its neighbour; the tests' rows are fixed and few.

Gradients (fp32 arithmetic, u = 2^-24): with S = r (|dz w| + |xh| mean|dz w xh|) for dx, every factor has a handful of
roundings and the mean D / 8 + 5 more: |error| <= (D / 8 + 24) u S, and half a step of the output's type.  dw sums T
terms in fp32, of a warp's rows one after another: |error| <= (rows a warp + 64) u sum |dz xh|.
"""
import numpy as np
import pytest

from oracle import attn as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module")
def q4q():
    import __graft_entry__
    __graft_entry__.build()
    import q4_quantized_matmul_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.set_device(0)
    return m


def heads_like(rng, *shape):
    return (rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)))).astype(np.float32)


def wide(*tensors):
    """Views [tokens, heads, D] of the rows of one tensor, as a fused projection writes them."""
    n = tensors[0].shape[0]
    buf = torch.cat([t.reshape(n, -1) for t in tensors], 1).cuda()
    out, at = [], 0
    for t in tensors:
        w = t.shape[1] * t.shape[2]
        out.append(buf[:, at: at + w].unflatten(1, t.shape[1:]))
        at += w
    return out


def rounded(x, type):
    """fp32 values rounded once to a type."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[type])


def same(got, want):
    """Equal values; NaN where NaN is."""
    return torch.equal(torch.nan_to_num(got.cpu().float(), nan=12345.0), torch.nan_to_num(want.float(), nan=12345.0))


@pytest.mark.parametrize("rot,base", [(16, 10000.0), (128, 500000.0), (64, 1.0)])
def test_table(q4q, rot, base):
    got = q4q.q4q_rope_table(5000, rot, base).cpu().numpy()
    want = ref.rope_table(5000, rot, base)
    assert np.all(np.abs(got.astype(np.float64) - want) <= np.spacing(np.abs(want)))
    assert np.mean(got != want) < 1e-3                          # 64-bit functions differ in their last bit


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (96, 96), (96, 48), (128, 128), (128, 112), (256, 256), (256, 32)])
@pytest.mark.parametrize("tokens,qh,kh", [(1, 32, 8), (5, 3, 1), (67, 7, 7)])
def test_norm_rope(q4q, mode, type, dim, rot, tokens, qh, kh):
    rng = np.random.default_rng([mode, dim, rot, tokens])
    q, k = (rounded(heads_like(rng, tokens, h, dim), type) for h in (qh, kh))
    qw, kw = ((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    table = ref.rope_table(300, rot)
    pos = rng.integers(0, 300, tokens).astype(np.int32)
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    for wq, wk, t in ((qw, kw, table), (qw, None, table), (None, None, table), (qw, kw, None)):
        gq, gk = q4q.q4q_qk_norm_rope(*wide(q, k), None if wq is None else cu(wq), None if wk is None else cu(wk), EPS,
                                      None if t is None else cu(t), cu(pos), mode)
        assert gq.dtype == TYPES[type] and gq.is_contiguous()
        for got, x, w in ((gq, q, wq), (gk, k, wk)):
            assert same(got, rounded(ref.norm_rope(x.double().numpy(), w, EPS, t, pos, mode == 1), type))
    # queries alone, in place, off a vector's alignment
    buf = torch.empty(q.numel() + 1, dtype=TYPES[type], device="cuda")
    mine = buf[1:].view(q.shape)
    mine.copy_(q)
    got, nothing = q4q.q4q_qk_norm_rope(mine, q_weight=cu(qw), eps=EPS, table=cu(table), pos=cu(pos), mode=mode, q_dst=mine)
    assert nothing is None and got.data_ptr() == mine.data_ptr()
    assert same(got, rounded(ref.norm_rope(q.double().numpy(), qw, EPS, table, pos, mode == 1), type))
    assert q4q.q4q_device_status() == 0


def test_norm_rope_of_many_tokens(q4q):
    """Work items of several rows, more of them than warps."""
    rng = np.random.default_rng(4)
    q, k = rounded(heads_like(rng, 1501, 11, 128), "f32"), rounded(heads_like(rng, 1501, 3, 128), "f32")
    w = (1 + 0.3 * rng.standard_normal(128)).astype(np.float32)
    table, pos = ref.rope_table(4096, 128), rng.integers(0, 4096, 1501).astype(np.int32)
    gq, gk = q4q.q4q_qk_norm_rope(q.cuda(), k.cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(w).cuda(), EPS, torch.from_numpy(table).cuda(),
                                  torch.from_numpy(pos).cuda())
    for got, x in ((gq, q), (gk, k)):
        want = ref.norm_rope(x.double().numpy(), w, EPS, table, pos, True).astype(np.float32)
        assert np.mean(got.cpu().numpy() != want) < 2e-4 and np.allclose(got.cpu().numpy(), want, rtol=2e-7, atol=0)


def test_sizes_of_rows(q4q):
    """Rows of zeros, of one value, of values far apart, tiny and large ones."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, 1, 64)).astype(np.float32)
    x[0] = 0
    x[1, 0, 1:] = 0
    x[2] *= 2.0 ** rng.integers(-40, 0, 64).astype(np.float32)
    x[3] *= 1e-12
    x[4] *= 1e15
    x[5] *= 2.0 ** 50
    w = np.ones(64, np.float32)
    for eps in (1e-6, 0.0, 1.0):
        rows = x[1:] if eps == 0.0 else x
        got, _ = q4q.q4q_qk_norm_rope(torch.from_numpy(rows).cuda(), q_weight=torch.from_numpy(w).cuda(), eps=eps)
        assert np.array_equal(got.cpu().numpy(), ref.norm_rope(rows, w, eps, None, None, True).astype(np.float32))


@pytest.mark.parametrize("mode", [0, 1])
def test_positions_outside_the_table(q4q, mode):
    rng = np.random.default_rng(6)
    x = torch.from_numpy(heads_like(rng, 5, 4, 64)).cuda()
    w = torch.ones(64, device="cuda")
    table = q4q.q4q_rope_table(100, 64)
    good = torch.tensor([3, 4, 5, 6, 7], dtype=torch.int32, device="cuda")
    bad = torch.tensor([3, 100, 5, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    want = q4q.q4q_qk_norm_rope(x, x, w, w, EPS, table, good, mode)
    back = q4q.q4q_qk_norm_rope_back(x, x, x, x, w, w, EPS, table, good, mode)
    assert q4q.q4q_device_status() == 0
    got = q4q.q4q_qk_norm_rope(x, x, w, w, EPS, table, bad, mode)
    for g, v in zip(got, want):
        assert torch.equal(g[[0, 2]], v[[0, 2]]) and not g[[1, 3, 4]].any()
    assert q4q.q4q_device_status() == 7
    gb = q4q.q4q_qk_norm_rope_back(x, x, x, x, w, w, EPS, table, bad, mode)
    for g, v in zip(gb[:2], back[:2]):
        assert torch.equal(g[[0, 2]], v[[0, 2]]) and not g[[1, 3, 4]].any()
    part = q4q.q4q_qk_norm_rope_back(*[x[[0, 2]].contiguous()] * 4, w, w, EPS, table, good[[0, 2]].contiguous(), mode)
    assert torch.allclose(gb[2], part[2], rtol=0, atol=1e-5) and torch.allclose(gb[3], part[3], rtol=0, atol=1e-5)
    assert q4q.q4q_device_status() == 7
    cache = torch.full((4 * q4q.q4q_kv_page_size(4, 64, 16),), 0x5A, dtype=torch.uint8, device="cuda")
    q4q.q4q_kv_append(cache, 16, x, x, torch.arange(5, dtype=torch.int32, device="cuda"), table=table, pos=bad, mode=mode)
    kept = cache.cpu().numpy()
    want = np.full(cache.numel(), 0x5A, np.uint8)
    xs = x.cpu().numpy()
    k = ref.norm_rope(xs, None, EPS, table.cpu().numpy(), np.where((bad.cpu().numpy() >= 0) & (bad.cpu().numpy() < 100), bad.cpu().numpy(), 0), mode == 1)
    ref.put(want, 16, [0, -1, 2, -1, -1], k.astype(np.float32), xs)
    assert np.array_equal(kept, want) and q4q.q4q_device_status() == 7


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,rot,tokens,qh,kh", [(64, 64, 1, 4, 2), (96, 48, 9, 5, 1), (128, 128, 700, 6, 2), (256, 256, 33, 3, 3), (64, 32, 5000, 8, 2)])
def test_gradients(q4q, mode, type, dim, rot, tokens, qh, kh):
    rng = np.random.default_rng([mode, dim, tokens])
    q, k, gq, gk = (rounded(heads_like(rng, tokens, h, dim), type) for h in (qh, kh, qh, kh))
    qw, kw = ((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    table, pos = ref.rope_table(300, rot), rng.integers(0, 300, tokens).astype(np.int32)
    cu = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()  # noqa: E731
    vq, vk = wide(q, k)
    out = q4q.q4q_qk_norm_rope_back(cu(gq), cu(gk), vq, vk, cu(qw), cu(kw), EPS, cu(table), cu(pos), mode)
    again = q4q.q4q_qk_norm_rope_back(cu(gq), cu(gk), vq, vk, cu(qw), cu(kw), EPS, cu(table), cu(pos), mode)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    u, eps_t = 2.0 ** -24, torch.finfo(TYPES[type]).eps
    for dx, dw, g, x, w in ((out[0], out[2], gq, q, qw), (out[1], out[3], gk, k, kw)):
        x64, g64 = x.double().numpy(), g.double().numpy()
        want, want_w = ref.norm_rope_back(g64, x64, w, EPS, table, pos, mode == 1)
        r = 1 / np.sqrt(np.mean(x64 ** 2, -1, keepdims=True) + EPS)
        a, b = ref.pairs(rot, mode == 1)
        size_z = np.abs(g64)
        both = np.abs(g64[..., a]) + np.abs(g64[..., b])
        size_z[..., a] = size_z[..., b] = both
        s = r * (size_z * np.abs(w) + np.abs(x64 * r) * np.mean(size_z * np.abs(w) * np.abs(x64 * r), -1, keepdims=True))
        assert np.all(np.abs(dx.double().cpu().numpy() - want) <= (dim / 8 + 24) * u * s + eps_t / 2 * np.abs(want) + 2.0 ** -25)
        rows = tokens * (qh + kh) / 8
        assert np.all(np.abs(dw.double().cpu().numpy() - want_w) <= (rows + 64) * u * (size_z * np.abs(x64 * r)).sum((0, 1)))
    # no weights: the rotation's transpose alone, and no key
    dq, dk, dqw, dkw = q4q.q4q_qk_norm_rope_back(cu(gq), None, vq, eps=EPS, table=cu(table), pos=cu(pos), mode=mode)
    assert dk is None and dqw is None and dkw is None
    assert same(dq, rounded(ref.turn(gq.double().numpy(), table, pos, mode == 1, back=True), type))


def test_gradients_against_differences(q4q):
    """<g, y(x + h e) - y(x - h e)> / 2h of the forward call in fp32; its roundings, 2^-22 of the sum of |g y|, are divided by
    2 h, and the third derivative adds h^2."""
    rng = np.random.default_rng(9)
    x, g = heads_like(rng, 3, 2, 64), rng.standard_normal((3, 2, 64)).astype(np.float32)
    w = (1 + 0.3 * rng.standard_normal(64)).astype(np.float32)
    table, pos = torch.from_numpy(ref.rope_table(50, 32)).cuda(), torch.tensor([1, 7, 49], dtype=torch.int32, device="cuda")
    cu = lambda v: torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda()  # noqa: E731
    dx, _, dw, _ = q4q.q4q_qk_norm_rope_back(cu(g), None, cu(x), None, cu(w), None, EPS, table, pos)

    def loss(x, w):
        y = q4q.q4q_qk_norm_rope(cu(x), None, cu(w), None, EPS, table, pos)[0].double().cpu().numpy()
        return (g * y).sum(), np.abs(g * y).sum()
    h = 2.0 ** -7
    for t, i, c in ((0, 0, 0), (1, 1, 40), (2, 0, 17)):
        e = np.zeros_like(x)
        e[t, i, c] = h * np.abs(x[t, i]).max()
        up, size = loss(x + e, w)
        step = ((x + e)[t, i, c].astype(np.float64) - (x - e)[t, i, c].astype(np.float64))
        got = (up - loss(x - e, w)[0]) / step
        assert abs(got - float(dx[t, i, c])) <= size * 2.0 ** -21 / step + 64 * h * h * np.abs(g[t, i]).max() / np.sqrt((x[t, i] ** 2).mean())
    for c in (3, 60):
        e = np.zeros_like(w)
        e[c] = h
        up, size = loss(x, w + e)
        step = (w + e)[c].astype(np.float64) - (w - e)[c].astype(np.float64)
        assert abs((up - loss(x, w - e)[0]) / step - float(dw[c])) <= size * 2.0 ** -21 / step


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,heads,page", [(64, 12, 16), (96, 3, 32), (128, 8, 64), (128, 1, 256), (256, 2, 16)])
@pytest.mark.parametrize("tokens", [1, 37])
def test_append_and_get(q4q, mode, type, dim, heads, page, tokens):
    """The bytes of the tokens' slots are the reference's, every other byte stays; rows come back exactly."""
    rng = np.random.default_rng([mode, dim, heads, tokens])
    k, v = (rounded(heads_like(rng, tokens, heads, dim), type) for _ in range(2))
    w = (1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)
    pages = tokens // page + 4
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    if tokens > 1:
        slots[[1, 5]] = [-1, -2 ** 31]
        slots[7] = pages * page - 1 if pages * page - 1 not in slots else slots[7]
    table, pos = ref.rope_table(300, dim // 2), rng.integers(0, 300, tokens).astype(np.int32)
    before = rng.integers(0, 256, pages * ref.page_size(heads, dim, page)).astype(np.uint8)
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    for weight, t in ((w, table), (None, table), (None, None), (w, None)):
        cache = cu(before.copy()).view(pages, -1)
        vk, vv = wide(k, v)
        got = q4q.q4q_kv_append(cache, page, vk, vv, cu(slots), None if weight is None else cu(weight), EPS, None if t is None else cu(t), cu(pos), mode)
        assert got.data_ptr() == cache.data_ptr()
        want = ref.put(before.copy(), page, slots, ref.norm_rope(k.double().numpy(), weight, EPS, t, pos, mode == 1).astype(np.float32),
                       v.float().numpy())
        assert np.array_equal(cache.cpu().numpy().reshape(-1), want)
    for dtype in TYPES:
        gk, gv = q4q.q4q_kv_get_rows(cache, page, heads, dim, cu(slots), dst_dtype=TYPES[dtype])
        rk, rv, _, _ = ref.get(want, page, heads, dim, np.maximum(slots, 0))
        for g, r in ((gk, rk), (gv, rv)):
            r = r.copy()
            r[slots < 0] = 0
            assert same(g, rounded(r.astype(np.float32), dtype))
    assert q4q.q4q_device_status() == 0


def test_append_of_special_values(q4q):
    """Zeros, ties, values past +-65504, infinities and NaN: block by block what the reference says."""
    x = np.zeros((8, 1, 128), np.float32)
    x[1, 0, :64] = np.arange(64) / 8 - 4                        # scale 1/2: quotients on half steps
    x[2, 0, :32] = 1e5
    x[2, 0, 32:64] = -3e38
    x[2, 0, 64] = 65504
    x[3, 0, 0], x[3, 0, 33], x[3, 0, 70] = np.inf, -np.inf, np.nan
    x[3, 0, 96:] = 1.0
    x[4, 0] = 1e-42
    x[5, 0] = 6e-8
    x[6, 0] = np.linspace(-1, 1, 128)
    x[7, 0] = -x[6, 0]
    cache = torch.zeros(q4q.q4q_kv_page_size(1, 128, 16), dtype=torch.uint8, device="cuda")
    slots = torch.arange(8, dtype=torch.int32, device="cuda")
    q4q.q4q_kv_append(cache, 16, torch.from_numpy(x).cuda(), torch.from_numpy(x[::-1].copy()).cuda(), slots)
    want = ref.put(np.zeros(cache.numel(), np.uint8), 16, range(8), x, x[::-1])
    got = cache.cpu().numpy()
    codes = 16 * 128
    assert np.array_equal(got[:codes], want[:codes])
    a, b = got[codes:].view(np.float16), want[codes:].view(np.float16)
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)]) and np.nanmax(a) == 8188


def test_slots_outside_the_cache(q4q):
    rng = np.random.default_rng(10)
    x = torch.from_numpy(heads_like(rng, 4, 2, 64)).cuda()
    cache = torch.full((2 * q4q.q4q_kv_page_size(2, 64, 16),), 0x33, dtype=torch.uint8, device="cuda")
    guard = cache.clone()
    slots = torch.tensor([32, 2 ** 31 - 1, 33, -7], dtype=torch.int32, device="cuda")
    q4q.q4q_kv_append(cache, 16, x, x, slots)
    assert torch.equal(cache, guard) and q4q.q4q_device_status() == 7
    k, v = q4q.q4q_kv_get_rows(cache, 16, 2, 64, slots)
    assert not k.any() and not v.any() and q4q.q4q_device_status() == 7
    k, v = q4q.q4q_kv_get_rows(cache, 16, 2, 64, slots[3:])
    assert not k.any() and not v.any() and q4q.q4q_device_status() == 0


def test_order_of_calls_and_graphs(q4q):
    """Each call reads what the one before it wrote into reused buffers, in a stream and in a replayed graph."""
    rng = np.random.default_rng(11)
    n, heads, dim, page = 6, 4, 128, 16
    table = q4q.q4q_rope_table(64, dim)
    w = torch.ones(dim, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda") + 3
    cache = torch.zeros(2 * q4q.q4q_kv_page_size(heads, dim, page), dtype=torch.uint8, device="cuda")
    src, q, k, v = (torch.empty(n, heads, dim, device="cuda") for _ in range(4))

    def step():
        q4q.q4q_qk_norm_rope(src, src, w, w, EPS, table, pos, 1, q, k)
        q4q.q4q_kv_append(cache, page, k, q, slots)
        q4q.q4q_kv_get_rows(cache, page, heads, dim, slots, k_dst=src, v_dst=v)
        q4q.q4q_qk_norm_rope(src, v, w, None, EPS, table, pos, 0, src, v)

    def want(x):
        t, p = table.cpu().numpy(), np.arange(n)
        y = ref.norm_rope(x, np.ones(dim), EPS, t, p, True).astype(np.float32)
        codes, d = ref.q4(y)
        z = ((codes.astype(np.float64) - 8) * d.astype(np.float64)[..., None]).reshape(y.shape)
        return ref.norm_rope(z, np.ones(dim), EPS, t, p, False).astype(np.float32), ref.norm_rope(z, None, EPS, t, p, False).astype(np.float32)
    torch.cuda.synchronize()
    graph = None
    for i in range(12):
        x = heads_like(rng, n, heads, dim)
        src.copy_(torch.from_numpy(x))
        if i == 6:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            src.copy_(torch.from_numpy(x))
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        a, b = want(x)
        assert np.array_equal(src.cpu().numpy(), a) and np.array_equal(v.cpu().numpy(), b)


def test_other_stream(q4q):
    rng = np.random.default_rng(12)
    x = torch.from_numpy(heads_like(rng, 50, 4, 64)).cuda()
    w = torch.ones(64, device="cuda")
    want = q4q.q4q_qk_norm_rope(x, x, w, w)
    back = q4q.q4q_qk_norm_rope_back(x, x, x, x, w, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q4q.q4q_qk_norm_rope(x, x, w, w, stream=side)
    gb = q4q.q4q_qk_norm_rope_back(x, x, x, x, w, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + gb, want + back))


def test_refusals(q4q):
    x, w = torch.zeros(4, 3, 64, device="cuda"), torch.ones(64, device="cuda")
    table, pos = q4q.q4q_rope_table(8, 64), torch.zeros(4, dtype=torch.int32, device="cuda")
    page = q4q.q4q_kv_page_size(3, 64, 16)
    cache = torch.zeros(page, dtype=torch.uint8, device="cuda")
    nr, ap, gr = q4q.q4q_qk_norm_rope, q4q.q4q_kv_append, q4q.q4q_kv_get_rows
    for error, call in (
            (TypeError, lambda: nr(x.cpu())), (TypeError, lambda: nr(x.double())), (ValueError, lambda: nr(x[0])),
            (ValueError, lambda: nr(x.transpose(0, 1))), (ValueError, lambda: nr(x[:, :, ::2])), (ValueError, lambda: nr(x[:1].expand(4, 3, 64))),
            (TypeError, lambda: nr(x, x.half())), (ValueError, lambda: nr(x, x[:3])), (ValueError, lambda: nr(x, None, w[:63])),
            (TypeError, lambda: nr(x, None, w.half())), (ValueError, lambda: nr(x, table=table)), (ValueError, lambda: nr(x, table=table, pos=pos[:3])),
            (TypeError, lambda: nr(x, table=table, pos=pos.long())), (q4q.Q4QError, lambda: nr(x, table=torch.zeros(8, 72, device="cuda"), pos=pos)),
            (q4q.Q4QError, lambda: nr(x, table=torch.zeros(8, 128, device="cuda"), pos=pos)), (q4q.Q4QError, lambda: nr(x, mode=2)),
            (q4q.Q4QError, lambda: nr(x, eps=-1.0)), (q4q.Q4QError, lambda: nr(torch.zeros(4, 3, 80, device="cuda"))),
            (TypeError, lambda: nr(x, q_dst=x.half())), (ValueError, lambda: nr(x, q_dst=x[:3].clone())),
            (ValueError, lambda: ap(cache[1:], 16, x, x, pos)), (q4q.Q4QError, lambda: ap(cache, 17, x, x, pos)), (q4q.Q4QError, lambda: ap(cache, 8, x, x, pos)),
            (ValueError, lambda: ap(cache, 16, x, x[:, :2], pos)), (TypeError, lambda: ap(cache, 16, x, x, pos.long())),
            (ValueError, lambda: ap(cache, 16, x, x, pos[:2])), (ValueError, lambda: gr(cache, 16, 4, 64, pos)), (q4q.Q4QError, lambda: gr(cache, 16, 3, 65, pos)),
            (TypeError, lambda: gr(cache, 16, 3, 64, pos, dst_dtype=torch.float64)), (q4q.Q4QError, lambda: q4q.q4q_rope_table(8, 24)),
            (q4q.Q4QError, lambda: q4q.q4q_rope_table(8, 32, 0.0))):
        with pytest.raises(error):
            call()
    assert nr(x[:0])[0].shape == (0, 3, 64)
    back = q4q.q4q_qk_norm_rope_back(x[:0], None, x[:0], None, w)
    assert back[0].shape == (0, 3, 64) and not back[2].any()
    ap(cache, 16, x[:0], x[:0], pos[:0])
    assert gr(cache, 16, 3, 64, pos[:0])[0].shape == (0, 3, 64)
    assert q4q.q4q_device_status() == 0
