"""Tokens sorted by expert and back, their gradients and the experts' products, against plain 64-bit forms.

Bars: places and copies are equal.  A weighted sum of top_k terms in fp32 is within
(top_k + 1) * 2^-24 of the sum of the terms' sizes, a dot product of ne0 terms within
(ne0 + 1) * 2^-24 of it, and each is then rounded to its type.  Products: as
test_gpu_mxfp4.py derives.
"""
import numpy as np
import pytest

from oracle import mx
from test_gpu_mxfp4 import TYPES, close, decoded_on_gpu, on_gpu, q4q, rand  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def choices(rng, n, top, experts, drop=0.1):
    ids = np.argsort(rng.random((n, experts)), axis=1)[:, :top] if top <= experts else rng.integers(0, experts, (n, top))
    return np.where(rng.random((n, top)) < drop, rng.choice([-1, experts, -2 ** 31, 2 ** 31 - 1], (n, top)), ids).astype(np.int32)


@pytest.mark.parametrize("n,top,experts", [(0, 2, 4), (1, 1, 1), (1, 2, 8), (3, 4, 7), (37, 4, 6), (511, 2, 1024), (1000, 8, 256),
                                           (8191, 4, 64), (40001, 2, 33), (70000, 8, 1024)])
def test_sort(q4q, n, top, experts):  # noqa: F811
    ids = choices(np.random.default_rng([n, top, experts]), n, top, experts)
    got = q4q.q4q_moe_sort(torch.from_numpy(ids).cuda(), experts)
    for name, a, b in zip(("first", "slot", "row"), got, mx.sort(ids, experts)):
        assert np.array_equal(a.cpu().numpy(), b), name


@pytest.mark.parametrize("fill", [-1, 0, 5, 63])
def test_sort_of_equal_ids(q4q, fill):  # noqa: F811
    ids = np.full((3000, 3), fill, np.int32)
    for a, b in zip(q4q.q4q_moe_sort(torch.from_numpy(ids).cuda(), 64), mx.sort(ids, 64)):
        assert np.array_equal(a.cpu().numpy(), b)


def plain_rows(ids, experts, x, rows, w, dy, dsorted):
    n, top = ids.shape
    first, slot, row = mx.sort(ids, experts)
    kept, out = first[-1], {}
    used = (row < kept).reshape(n, top)
    at = row.reshape(n, top)
    r0, d0 = rows.copy(), dsorted.copy()
    r0[kept:], d0[kept:] = 0.0, 0.0
    w0 = np.where(used, w, 0.0)
    out["sorted"] = np.zeros((n * top, x.shape[1]))
    out["sorted"][at[used]] = np.repeat(x[:, None], top, 1)[used]
    out["y"] = (w0[..., None] * r0[at]).sum(1)
    out["y_size"] = np.abs(w0[..., None] * r0[at]).sum(1)
    out["drows"] = np.zeros((n * top, x.shape[1]))
    out["drows"][at[used]] = (w0[..., None] * dy[:, None])[used]
    out["dw"] = np.where(used, (r0[at] * dy[:, None]).sum(-1), 0.0)
    out["dw_size"] = np.abs(r0[at] * dy[:, None]).sum(-1)
    out["dx"] = np.where(used[..., None], d0[at], 0.0).sum(1)
    out["dx_size"] = np.where(used[..., None], np.abs(d0[at]), 0.0).sum(1)
    return out, kept


@pytest.mark.parametrize("type_", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,top,experts,ne0", [(1, 2, 8, 4096), (5, 1, 3, 1), (37, 4, 6, 77), (129, 2, 40, 264), (700, 8, 16, 1000), (60, 3, 5, 2050)])
def test_rows_and_gradients(q4q, type_, n, top, experts, ne0):  # noqa: F811
    rng = np.random.default_rng([n, top, ne0])
    ids = choices(rng, n, top, experts)
    x, xv = on_gpu(rng.standard_normal((n, ne0)), type_)
    rows, rv = on_gpu(rng.standard_normal((n * top, ne0)), type_)
    dy, dv = on_gpu(rng.standard_normal((n, ne0)), type_)
    ds, sv = on_gpu(rng.standard_normal((n * top, ne0)), type_)
    w, wv = on_gpu(rng.standard_normal((n, top)), "f32")
    ref, kept = plain_rows(ids, experts, xv, rv, wv, dv, sv)
    rows[kept:], ds[kept:] = float("nan"), float("inf")       # rows of no expert are not read
    w[torch.from_numpy((ids < 0) | (ids >= experts)).cuda()] = float("nan")
    first, slot, row = q4q.q4q_moe_sort(torch.from_numpy(ids).cuda(), experts)
    u = TYPES[type_][1]
    tiny = 2.0 ** -25 if type_ == "f16" else 0.0

    def near(got, name, terms, unit):
        got, r = got.double().cpu().numpy(), ref[name]
        size = ref.get(name + "_size", np.abs(r))
        assert (np.abs(got - r) <= (terms + 1) * 2.0 ** -24 * size + unit * np.abs(r) + tiny).all(), name
    assert np.array_equal(q4q.q4q_moe_gather(x, first, row, top).double().cpu().numpy(), ref["sorted"])
    near(q4q.q4q_moe_gather_back(ds, first, row, top), "dx", top, u * 1.01)
    near(q4q.q4q_moe_combine(rows, first, row, w), "y", top, u * 1.01)
    drows, dw = q4q.q4q_moe_combine_back(dy, rows, first, row, w)
    near(drows, "drows", 1, u * 1.01)
    near(dw, "dw", ne0, 2.0 ** -24)


def test_gradients_by_differences(q4q):  # noqa: F811
    """L = <dy, combine(rows, w)> is linear in rows and in w, so a central difference of any
    step is its derivative but for rounding: with steps of 1 and sums of at most 4 terms of
    size under 32 in fp32, and the outer sum in 64 bits, under 600 * 5 * 2^-24 * 32 * 2."""
    rng = np.random.default_rng(21)
    n, top, experts, ne0 = 6, 3, 4, 100
    ids = torch.from_numpy(choices(rng, n, top, experts, 0.2)).cuda()
    first, slot, row = q4q.q4q_moe_sort(ids, experts)
    rows = torch.from_numpy(rng.standard_normal((n * top, ne0)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.standard_normal((n, top)).astype(np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((n, ne0)).astype(np.float32)).cuda()
    drows, dw = q4q.q4q_moe_combine_back(dy, rows, first, row, w)
    dx_in = torch.from_numpy(rng.standard_normal((n * top, ne0)).astype(np.float32)).cuda()
    dx = q4q.q4q_moe_gather_back(dx_in, first, row, top)
    tol = 600 * 5 * 2.0 ** -24 * 32 * 2

    def loss(r, v):
        return float((dy.double() * q4q.q4q_moe_combine(r, first, row, v).double()).sum())
    for t in range(n):
        for j in range(top):
            a, b = w.clone(), w.clone()
            a[t, j] += 1
            b[t, j] -= 1
            assert abs((loss(rows, a) - loss(rows, b)) / 2 - float(dw[t, j])) <= tol
    for r, c in [(0, 0), (3, 99), (n * top - 1, 5), (7, 50)]:
        a, b = rows.clone(), rows.clone()
        a[r, c] += 1
        b[r, c] -= 1
        assert abs((loss(a, w) - loss(b, w)) / 2 - float(drows[r, c])) <= tol
    x = torch.from_numpy(rng.standard_normal((n, ne0)).astype(np.float32)).cuda()
    kept = int(first[-1])
    for t, c in [(0, 0), (5, 99), (2, 17)]:
        a, b = x.clone(), x.clone()
        a[t, c] += 1
        b[t, c] -= 1
        d = (q4q.q4q_moe_gather(a, first, row, top).double() - q4q.q4q_moe_gather(b, first, row, top).double())[:kept]
        assert abs(float((dx_in.double()[:kept] * d).sum()) / 2 - float(dx[t, c])) <= tol


def experts_product(q4q, n, top, experts, rows, k, acts, type_, ids=None, sorted_rows=False, **more):  # noqa: F811
    rng = np.random.default_rng([n, top, experts, rows, k])
    ids = choices(rng, n, top, experts) if ids is None else ids
    packs = [mx.pack(rand(rng, rows, k, 0.05).astype(np.float32)) for _ in range(experts)]
    w = torch.from_numpy(np.stack([p[0] for p in packs])).cuda()
    x, v = on_gpu(rand(rng, n * top if sorted_rows else n, k), type_)
    e = mx.encode(v, acts)[2]
    order = q4q.q4q_moe_sort(torch.from_numpy(ids).cuda(), experts)
    got = q4q.q4q_mul_mat_id_mxfp4(w, k, rows, x, order[0], None if sorted_rows else order[1], top, int(acts == "mxfp8"), **more)
    first, slot, _ = mx.sort(ids, experts)
    ref, size = np.zeros((n * top, rows)), np.zeros((n * top, rows))
    for j in range(experts):
        r = np.arange(first[j], first[j + 1])
        a = e[r] if sorted_rows else e[slot[r] // top]
        ref[r], size[r] = a @ packs[j][1].T, np.abs(a) @ np.abs(packs[j][1]).T
    return got, ref, size


@pytest.mark.parametrize("acts", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("n,top,experts,rows,k", [(1, 1, 1, 1, 32), (1, 2, 8, 300, 512), (3, 2, 8, 257, 4096), (20, 4, 5, 128, 96),
                                                  (100, 2, 3, 777, 1504), (517, 4, 32, 140, 288), (300, 1, 2, 260, 256),
                                                  (64, 2, 1024, 33, 64), (900, 2, 4, 300, 256)])
def test_experts_products(q4q, n, top, experts, rows, k, acts):  # noqa: F811
    got, ref, size = experts_product(q4q, n, top, experts, rows, k, acts, "f32")
    close(got, ref, size, k, "f32")
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("n,top,experts,rows,k,acts", [(150, 2, 4, 5000, 1056, "mxfp8"), (80, 2, 4, 9000, 2048, "mxfp8"), (600, 2, 3, 5000, 1056, "mxfp4"),
                                                       (450, 2, 4, 3000, 2048, "mxfp8"), (2, 3, 9, 700, 3104, "mxfp8")])
def test_experts_products_of_large_matrices(q4q, n, top, experts, rows, k, acts):  # noqa: F811
    """Sizes at which tiles are taken by pairs of CTAs and by clusters; one expert has a third of the choices."""
    rng = np.random.default_rng([n, rows, k])
    ids = choices(rng, n, top, experts)
    ids[: n // 3, 0] = experts - 1
    w, values = zip(*[decoded_on_gpu(q4q, rng, rows, k) for _ in range(experts)])
    x, v = on_gpu(rand(rng, n, k), "f32")
    e = torch.from_numpy(mx.encode(v, acts)[2]).cuda()
    order = q4q.q4q_moe_sort(torch.from_numpy(ids).cuda(), experts)
    got = q4q.q4q_mul_mat_id_mxfp4(torch.stack(w), k, rows, x, order[0], order[1], top, int(acts == "mxfp8"))
    first, slot, _ = mx.sort(ids, experts)
    ref, size = torch.zeros(n * top, rows, dtype=torch.float64, device="cuda"), torch.zeros(n * top, rows, dtype=torch.float64, device="cuda")
    for j in range(experts):
        r = slice(int(first[j]), int(first[j + 1]))
        a = e[torch.from_numpy(slot[r].astype(np.int64) // top).cuda()]
        ref[r], size[r] = a @ values[j].T, a.abs() @ values[j].abs().T
    close(got, ref.cpu().numpy(), size.cpu().numpy(), k, "f32")


@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_experts_products_of_sorted_rows(q4q, type_):  # noqa: F811
    got, ref, size = experts_product(q4q, 77, 2, 6, 200, 320, "mxfp8", type_, sorted_rows=True)
    assert got.dtype == TYPES[type_][0]
    close(got, ref, size, 320, type_)


def test_experts_products_of_uneven_shares(q4q):  # noqa: F811
    one = np.zeros((500, 2), np.int32)
    one[:, 1] = 3                                              # two experts have everything
    none = np.full((40, 2), -1, np.int32)                      # nobody has anything
    last = np.full((40, 2), -1, np.int32)
    last[39, 1] = 7                                            # one row, at the last expert
    for ids in (one, none, last):
        got, ref, size = experts_product(q4q, ids.shape[0], 2, 8, 260, 288, "mxfp4", "f32", ids=ids)
        close(got, ref, size, 288, "f32")


def test_experts_products_stay_in_bounds_of_a_bad_first(q4q):  # noqa: F811
    """Whatever stands in `first`, rows are clamped to those there are (every access is bounded by the kernels' own checks)."""
    rng = np.random.default_rng(31)
    w = torch.from_numpy(np.stack([mx.pack(rand(rng, 64, 64).astype(np.float32))[0] for _ in range(4)])).cuda()
    x = torch.randn(10, 64, device="cuda")
    slot = torch.arange(10, dtype=torch.int32, device="cuda")
    for first in ([0, 50, -7, 3, 10], [9, 0, 9, 0, 9], [-5, -5, 100, 100, 1000], [2 ** 31 - 1] * 5):
        f = torch.tensor(first, dtype=torch.int32, device="cuda")
        q4q.q4q_mul_mat_id_mxfp4(w, 64, 64, x, f, slot, 1)
        assert q4q.q4q_device_status() == 0


def test_the_example_runs(q4q):  # noqa: F811
    """Against fp32 activations on the same weights: E4M3 rounds by at most 2^-4 of a value, 2^-4 / sqrt(3) = 0.036 in
    the root mean square where it rounds worst, independently along K.  x is rounded once and enters as gate (slope of
    silu under 1.1) and up, the product is rounded again: (1.1 + 1 + 1) * 0.036 = 0.112, and the largest elements of
    blocks that saturate at 448 and the bf16 roundings between the steps add under 0.02."""
    from examples import moe_ffn_mxfp4
    assert moe_ffn_mxfp4.main(tokens=33, hidden=256, ff=512, experts=8, top=2) < 0.132


def test_rows_whose_offsets_pass_32_bits(q4q):  # noqa: F811
    """540,000 sorted rows of 4096: 2.2e9 values.  Halves and doubles of fp16 normals are exact."""
    n, top, ne0 = 270000, 2, 4096
    g = torch.Generator(device="cuda").manual_seed(16)
    x = torch.randint(1, 1000, (n, ne0), generator=g, device="cuda", dtype=torch.int16).half()
    ids = torch.stack([torch.randint(0, 4, (n,), generator=g, device="cuda"), torch.randint(4, 7, (n,), generator=g, device="cuda")], 1).int()
    first, slot, row = q4q.q4q_moe_sort(ids, 7)
    rows = q4q.q4q_moe_gather(x, first, row, top)
    tail = slot[-1000:].long() // top
    assert torch.equal(rows[-1000:], x[tail])
    w = torch.full((n, top), 0.5, device="cuda")
    assert torch.equal(q4q.q4q_moe_combine(rows, first, row, w), x)
    assert torch.equal(q4q.q4q_moe_gather_back(rows, first, row, top), x * 2)
    drows, dw = q4q.q4q_moe_combine_back(x, rows, first, row, w)
    assert torch.equal(drows[-1000:], x[tail] / 2)
    square = (x[-1000:].double() ** 2).sum(1)
    assert ((dw[-1000:].double() - square[:, None]).abs() <= (ne0 + 1) * 2.0 ** -24 * square[:, None]).all()


def test_experts_outputs_whose_offsets_pass_32_bits(q4q):  # noqa: F811
    """40,000 rows of 60,000 outputs: 2.4e9."""
    n, top, experts, rows, k = 20000, 2, 3, 60000, 32
    rng = np.random.default_rng(17)
    w, values = zip(*(decoded_on_gpu(q4q, rng, rows, k, 0.05) for _ in range(experts)))
    x, v = on_gpu(rand(rng, n, k), "bf16")
    ids = choices(rng, n, top, experts, drop=0.0)
    first, slot, _ = q4q.q4q_moe_sort(torch.from_numpy(ids).cuda(), experts)
    y = q4q.q4q_mul_mat_id_mxfp4(torch.stack(w), k, rows, x, first, slot, top)
    at = slot[-300:].long() // top                            # of the last expert
    assert int(first[experts - 1]) <= n * top - 300
    e = mx.encode(v, "mxfp8")[2][at.cpu().numpy()]
    m = values[experts - 1].cpu().numpy()
    close(y[-300:], e @ m.T, np.abs(e) @ np.abs(m).T, k, "bf16")
    assert q4q.q4q_device_status() == 0
