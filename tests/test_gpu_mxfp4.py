"""MXFP4 matrices and their products on the GPU against the plain 64-bit reference.

Bars:
  * encoder: every byte equal; row gather: equal.
  * products: the codes and scales of both sides are the reference's, and a product of two
    elements is exact, so only the fp32 sums differ.  A tensor core adds at least one block
    (32 products) at a time: products and running sum are aligned to the largest of them
    and cut at 24 bits or more, 33 terms, so one addition is off by at most 33 * 2^-24 of
    the largest term, at most 33 * 2^-24 * S with S = sum_k |w_k x_k|; in all K / 32 + 1 of
    them, counting joins of split sums (at most K / 128).  The bound below takes the mean
    size of the running sum, not its largest, as S / 2, drops no term, and adds half a unit
    of the output's type: (K / 32 + K / 128 + 2) * 2^-23 * S + u * |ref|.
"""
import numpy as np
import pytest

from oracle import mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, 2.0 ** -24), "f16": (torch.float16, 2.0 ** -11), "bf16": (torch.bfloat16, 2.0 ** -8)}


@pytest.fixture(scope="module")
def q4q():
    import __graft_entry__
    __graft_entry__.build()
    import q4_quantized_matmul_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.set_device(0)
    return m


def rand(rng, rows, k, scale=1.0):
    x = rng.standard_normal((rows, k)) * scale
    x *= np.where(rng.random(k) < 0.02, 10.0, 1.0)
    b = x.reshape(rows, -1, 32)
    b[rng.random(b.shape[:2]) < 0.05] = 0.0
    return x


def on_gpu(x, type_):
    """x rounded to the type, on the GPU and as float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TYPES[type_][0]).cuda()
    return t, t.double().cpu().numpy()


def close(got, ref, size, k, type_, what=""):
    got = got.double().cpu().numpy()
    tol = (k / 32 + k / 128 + 2) * 2.0 ** -23 * size + TYPES[type_][1] * np.abs(ref) + (2.0 ** -25 if type_ == "f16" else 0.0)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %g" % (what, bad.sum(), bad.size, np.abs(got - ref)[bad].max())


# ------------------------------------------------------------------ encoder --

@pytest.mark.parametrize("type_", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 32), (5, 96), (127, 256), (129, 288), (40, 4096), (300, 1504)])
def test_encoder_bytes(q4q, type_, rows, k):
    x, v = on_gpu(rand(np.random.default_rng([rows, k]), rows, k), type_)
    assert np.array_equal(q4q.q4q_quantize_mxfp4(x).cpu().numpy(), mx.pack(v)[0])


def special_rows():
    grid = np.concatenate((mx.E2M1, (mx.E2M1[1:] + mx.E2M1[:-1]) / 2, [5.999, 6.5, 7.0, 7.999, 4.0, 2.0 ** -20, 0.0, 1.0]))
    rows = [np.resize(np.concatenate((grid, -grid)) * 2.0 ** e, 64) for e in (-140, -127, -126, -125, -124, -60, 0, 1, 90, 124)]
    rows += [np.full(64, 3.4028234e38), np.full(64, -0.0), np.full(64, 2.0 ** -149), np.full(64, 1.9999999 * 2.0 ** -126)]
    for i, v in ((3, np.inf), (40, -np.inf), (63, np.nan)):
        r = np.linspace(-3, 3, 64)
        r[i] = v
        rows.append(r)
    return np.array(rows).astype(np.float32)


def test_encoder_special_values_and_row_gather(q4q):
    x, v = on_gpu(special_rows(), "f32")
    packed, values = mx.pack(v)
    w = q4q.q4q_quantize_mxfp4(x)
    assert np.array_equal(w.cpu().numpy(), packed)
    got = q4q.q4q_get_rows_mxfp4(w, 64, len(v)).cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(values))
    assert np.array_equal(got[~np.isnan(got)], values.astype(np.float32)[~np.isnan(got)])


def test_encoder_takes_unaligned_rows_and_several_matrices(q4q):
    x, v = on_gpu(rand(np.random.default_rng(3), 3 * 70, 160).reshape(-1), "f16")
    odd = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:]
    odd.copy_(x)
    w = q4q.q4q_quantize_mxfp4(odd.view(3, 70, 160)).cpu().numpy()
    for m in range(3):
        assert np.array_equal(w[m], mx.pack(v.reshape(3, 70, 160)[m])[0])


def at_offset(t, offset):
    """t in memory that starts `offset` elements behind a 256-byte boundary."""
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:]
    return buf.copy_(t.reshape(-1)).view(t.shape)


@pytest.mark.parametrize("type_,offset", [("f32", 1), ("f32", 4), ("f32", 8), ("f16", 3), ("f16", 8), ("f16", 16), ("bf16", 1), ("bf16", 8), ("bf16", 16)])
def test_encoders_of_rows_at_any_offset(q4q, type_, offset):
    x, v = on_gpu(special_rows() if type_ == "f32" else rand(np.random.default_rng(5), 21, 64), type_)
    assert np.array_equal(q4q.q4q_quantize_mxfp4(at_offset(x, offset)).cpu().numpy(), mx.pack(v)[0])
    rng = np.random.default_rng([6, offset])
    w = torch.from_numpy(mx.pack(rand(rng, 200, 352, 0.02).astype(np.float32))[0]).cuda()
    x = on_gpu(rand(rng, 11, 352), type_)[0]
    for acts in (0, 1):
        assert torch.equal(q4q.q4q_mul_mat_mxfp4(w, 352, 200, at_offset(x, offset), acts), q4q.q4q_mul_mat_mxfp4(w, 352, 200, x, acts))


@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_encoder_infinities_and_nan_of_16_bit_types(q4q, type_):
    """Wherever in a block they stand, with either sign."""
    x = rand(np.random.default_rng(7), 128, 64)
    for r in range(128):
        x[r, r % 64] = [np.inf, -np.inf, np.nan][r % 3]
    x, v = on_gpu(x, type_)
    packed, values = mx.pack(v)
    w = q4q.q4q_quantize_mxfp4(x)
    assert np.array_equal(w.cpu().numpy(), packed)
    assert np.array_equal(np.isnan(q4q.q4q_get_rows_mxfp4(w, 64, 128).cpu().numpy()), np.isnan(values))


def test_row_gather_ids(q4q):
    x, v = on_gpu(rand(np.random.default_rng(4), 300, 288), "bf16")
    values = mx.pack(v)[1].astype(np.float32)
    w = q4q.q4q_quantize_mxfp4(x)
    ids = np.array([299, 0, 0, 128, 127, 17], np.int32)
    got = q4q.q4q_get_rows_mxfp4(w, 288, 300, torch.from_numpy(ids).cuda())
    assert np.array_equal(got.cpu().numpy(), values[ids])
    bad = q4q.q4q_get_rows_mxfp4(w, 288, 300, torch.tensor([5, -1, 300], dtype=torch.int32, device="cuda")).cpu().numpy()
    assert q4q.q4q_device_status() == 7 and q4q.q4q_device_status() == 0
    assert np.array_equal(bad[0], values[5]) and not bad[1:].any()


# ----------------------------------------------------------------- products --

def product(q4q, rows, k, tokens, acts, type_, seed=0, dst=None, **more):
    rng = np.random.default_rng([rows, k, tokens, seed])
    packed, w = mx.pack(rand(rng, rows, k, 0.02).astype(np.float32))
    x, v = on_gpu(rand(rng, tokens, k), type_)
    e = mx.encode(v, acts)[2]
    got = q4q.q4q_mul_mat_mxfp4(torch.from_numpy(packed).cuda(), k, rows, x, int(acts == "mxfp8"), dst_dtype=dst, **more)
    return got, e @ w.T, np.abs(e) @ np.abs(w).T


@pytest.mark.parametrize("acts", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 100, 128, 129, 256, 257, 300])
def test_product_token_counts(q4q, tokens, acts):
    got, ref, size = product(q4q, 261, 544, tokens, acts, "f32")
    close(got, ref, size, 544, "f32", "%d tokens" % tokens)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("acts", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows,k,tokens", [(1, 32, 1), (1, 4096, 1), (31, 32, 5), (128, 14336, 3), (127, 96, 40), (129, 256, 12),
                                           (777, 1504, 21), (2000, 2048, 1), (40000, 64, 2), (4100, 768, 200), (100, 7200, 70),
                                           (128, 4096, 1000), (20000, 256, 300)])
def test_product_shapes(q4q, rows, k, tokens, acts):
    got, ref, size = product(q4q, rows, k, tokens, acts, "f32")
    close(got, ref, size, k, "f32")


def decoded_on_gpu(q4q, rng, rows, k, scale=0.02):
    """A large MXFP4 matrix and its values in 64 bits on the GPU, by way of the encoder and the row gather."""
    w = q4q.q4q_quantize_mxfp4(torch.from_numpy(rand(rng, rows, k, scale).astype(np.float32)).cuda())
    return w, q4q.q4q_get_rows_mxfp4(w, k, rows).double()


@pytest.mark.parametrize("rows,k,tokens,acts", [(19400, 2048, 100, "mxfp8"), (19400, 2048, 128, "mxfp4"), (20000, 4096, 50, "mxfp8"),
                                                (9700, 1024, 300, "mxfp4"), (9700, 1024, 520, "mxfp8"), (9601, 1056, 257, "mxfp8"),
                                                (3000, 5056, 1, "mxfp8"), (1000, 2080, 60, "mxfp4"), (40000, 288, 64, "mxfp8")])
def test_product_of_large_matrices(q4q, rows, k, tokens, acts):
    """Sizes at which tiles are taken by pairs of CTAs, by clusters, and in several rounds."""
    rng = np.random.default_rng([rows, k, tokens])
    w, values = decoded_on_gpu(q4q, rng, rows, k)
    x, v = on_gpu(rand(rng, tokens, k), "f32")
    e = torch.from_numpy(mx.encode(v, acts)[2]).cuda()
    got = q4q.q4q_mul_mat_mxfp4(w, k, rows, x, int(acts == "mxfp8"))
    close(got, (e @ values.T).cpu().numpy(), (e.abs() @ values.abs().T).cpu().numpy(), k, "f32")


@pytest.mark.parametrize("acts", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("type_,dst", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_product_types(q4q, type_, dst, acts):
    for tokens in (3, 70):
        got, ref, size = product(q4q, 300, 1056, tokens, acts, type_, dst=TYPES[dst][0])
        assert got.dtype == TYPES[dst][0]
        close(got, ref, size, 1056, dst)


def test_product_of_unaligned_rows_and_a_filled_workspace(q4q):
    rng = np.random.default_rng(8)
    packed, w = mx.pack(rand(rng, 200, 320).astype(np.float32))
    x, v = on_gpu(rand(rng, 9, 320), "bf16")
    odd = torch.empty(x.numel() + 3, dtype=x.dtype, device="cuda")[3:].view(9, 320)
    odd.copy_(x)
    dst = torch.empty(9 * 200 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(9, 200)
    ws = torch.full((q4q.q4q_mul_mat_mxfp4_workspace_size(320, 200, 9),), 255, dtype=torch.uint8, device="cuda")
    wd = torch.from_numpy(packed).cuda()
    q4q.q4q_mul_mat_mxfp4(wd, 320, 200, odd, dst=dst, workspace=ws)
    e = mx.encode(v, "mxfp8")[2]
    close(dst, e @ w.T, np.abs(e) @ np.abs(w).T, 320, "bf16")
    with pytest.raises(q4q.Q4QError):
        q4q.q4q_mul_mat_mxfp4(wd, 320, 200, odd, workspace=ws[:-256])
    with pytest.raises(ValueError):
        q4q.q4q_mul_mat_mxfp4(wd, 320, 200, x[:, ::2])
    with pytest.raises(ValueError):
        q4q.q4q_mul_mat_mxfp4(wd[:-1], 320, 200, x)


def test_product_repeats_to_the_bit(q4q):
    for rows, k, tokens in ((128, 14336, 3), (4096, 4096, 1), (1000, 8192, 130)):
        a = [product(q4q, rows, k, tokens, "mxfp8", "f32")[0] for _ in range(3)]
        assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])


def test_product_nan_blocks_reach_their_outputs_only(q4q):
    rng = np.random.default_rng(9)
    wv, xv = rand(rng, 150, 512).astype(np.float32), rand(rng, 40, 512).astype(np.float32)
    wv[70, 33], xv[5, 400], xv[6, 0] = np.inf, np.nan, -np.inf
    packed, w = mx.pack(wv)
    for acts in ("mxfp4", "mxfp8"):
        got = q4q.q4q_mul_mat_mxfp4(torch.from_numpy(packed).cuda(), 512, 150, torch.from_numpy(xv).cuda(), int(acts == "mxfp8"))
        ref = mx.encode(xv, acts)[2] @ w.T
        assert np.array_equal(np.isnan(got.cpu().numpy()), np.isnan(ref))
        assert np.isnan(ref[5]).all() and np.isnan(ref[:, 70]).all() and np.isnan(ref).sum() == 2 * 150 + 38


def test_product_scales_at_the_ends_of_their_range(q4q):
    rng = np.random.default_rng(10)
    for ew, ex in ((-100, 110), (100, -120), (120, -30), (-60, -40)):
        packed, w = mx.pack((rand(rng, 130, 288) * 2.0 ** ew).astype(np.float32))
        x, v = on_gpu(rand(rng, 20, 288) * 2.0 ** ex, "f32")
        e = mx.encode(v, "mxfp8")[2]
        got = q4q.q4q_mul_mat_mxfp4(torch.from_numpy(packed).cuda(), 288, 130, x)
        close(got, e @ w.T, np.abs(e) @ np.abs(w).T, 288, "f32", "2^%d x 2^%d" % (ew, ex))


def test_product_on_another_stream_and_chained(q4q):
    rng = np.random.default_rng(11)
    packed, w = mx.pack(rand(rng, 256, 256, 0.05).astype(np.float32))
    wd = torch.from_numpy(packed).cuda()
    x, v = on_gpu(rand(rng, 4, 256), "f32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = x
    for _ in range(8):                                        # each call reads the last one's result
        y = q4q.q4q_mul_mat_mxfp4(wd, 256, 256, y, stream=side, flags=q4q.Q4Q_MUL_MAT_PDL)
    z = x
    for _ in range(8):
        z = q4q.q4q_mul_mat_mxfp4(wd, 256, 256, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z)


def test_results_on_another_stream_take_no_memory_of_this_one(q4q):
    """A tensor freed here may still be read by work in flight here."""
    rng = np.random.default_rng(14)
    wd = torch.from_numpy(mx.pack(rand(rng, 5000, 256, 0.05).astype(np.float32))[0]).cuda()
    x = on_gpu(rand(rng, 1000, 256), "f32")[0]
    ref = q4q.q4q_mul_mat_mxfp4(wd, 256, 5000, x)
    old = torch.empty_like(ref)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    at, size = old.data_ptr(), old.numel() * 4
    del old
    got = q4q.q4q_mul_mat_mxfp4(wd, 256, 5000, x, stream=side)
    assert got.data_ptr() + size <= at or at + size <= got.data_ptr()
    side.synchronize()
    assert torch.equal(got, ref)
    with pytest.raises(ValueError):                           # nor a copy made here
        q4q.q4q_mul_mat_mxfp4(wd, 256, 5000, x.view(2, 500, 256)[:, ::2], stream=side)
    assert torch.equal(q4q.q4q_mul_mat_mxfp4(wd, 256, 5000, x.view(2, 500, 256)), ref)


def test_product_in_a_graph(q4q):
    rng = np.random.default_rng(12)
    packed, w = mx.pack(rand(rng, 500, 1024, 0.05).astype(np.float32))
    wd, x = torch.from_numpy(packed).cuda(), on_gpu(rand(rng, 3, 1024), "bf16")[0]
    ref = q4q.q4q_mul_mat_mxfp4(wd, 1024, 500, x)
    dst = torch.zeros_like(ref)
    ws = torch.empty(q4q.q4q_mul_mat_mxfp4_workspace_size(1024, 500, 3), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4q.q4q_mul_mat_mxfp4(wd, 1024, 500, x, dst=dst, workspace=ws)
    for _ in range(3):
        dst.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dst, ref)


def test_product_wait_that_runs_out(q4q):
    rng = np.random.default_rng(13)
    wd = torch.from_numpy(mx.pack(rand(rng, 300, 4096).astype(np.float32))[0]).cuda()
    for tokens in (1, 40, 300):
        for acts in (0, 1):
            x = torch.randn(tokens, 4096, device="cuda")
            q4q.q4q_debug_mul_mat_mxfp4_timeout(wd, 4096, 300, x, acts, 2_000_000)
            assert q4q.q4q_device_status() == 6
            a = q4q.q4q_mul_mat_mxfp4(wd, 4096, 300, x, acts)
            assert q4q.q4q_device_status() == 0 and torch.isfinite(a).all()


def test_matrix_whose_offsets_pass_32_bits(q4q):
    """1,100,000 rows of 4096: 9 GB of bf16, 2.2 GB of codes; what stands in its last rows comes out there."""
    rows, k, last = 1100000, 4096, 200
    rng = np.random.default_rng(15)
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    tail, v = on_gpu(rand(rng, last, k, 0.02), "bf16")
    x[-last:] = tail
    w = q4q.q4q_quantize_mxfp4(x)
    del x, tail
    values = mx.pack(v)[1]
    n = 270000                                                # 4.4 GB of fp32
    got = q4q.q4q_get_rows_mxfp4(w, k, rows, torch.arange(rows - n, rows, dtype=torch.int32, device="cuda"))
    assert np.array_equal(got[-last:].cpu().numpy(), values.astype(np.float32)) and not got[:-last].any()
    del got
    t, u = on_gpu(rand(rng, 2, k), "f32")
    e = mx.encode(u, "mxfp8")[2]
    y = q4q.q4q_mul_mat_mxfp4(w, k, rows, t)
    close(y[:, -last:], e @ values.T, np.abs(e) @ np.abs(values).T, k, "f32")
    assert not y[:, :-last].any() and q4q.q4q_device_status() == 0


@pytest.mark.parametrize("acts", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows,k,tokens", [(100, 4096, 12), (100, 4096, 30), (4500, 4096, 16), (4500, 4096, 25), (800, 20992, 660)])
def test_product_of_long_rows(q4q, rows, k, tokens, acts):
    """Sizes at which clusters share the K of tiles of 16 and 32 tokens, and pairs take tiles of 64."""
    test_product_of_large_matrices(q4q, rows, k, tokens, acts)
