"""Attention over the paged 4-bit cache against oracle/attn.py (numpy, 64 bits).

Bounds, of the form that keeps fp32 throughout.  u = 2^-24.  Queries and weights are two fp16 each, so
within 2^-22 of themselves; codes and scales are exact.
 - A score is sum_b d_b (sum q code - 8 sum q): every term and partial sum is at most the sum of |q| 8 d (codes
   reach 15, less 8: 16 with the offset, twice that), over 2 MMAs, D / 32 blocks and the roundings beside them.  With
   `span` = |scale| sum |q| 8 d and a sum in the tensor cores taken to 2^-22 (they may cut instead of round):
   |score's error| <= span (2 + 2 (D / 32 + 4)) 2^-22 =: e.
 - A weight is off by a factor exp(2 e) at most against the others, by 2^-21 of exp2 and its operand's rounding (an
   operand of up to `span` log2 e in size adds span 2^-23), by 2^-22 of its two halves.
 - An output sums weights times values, each at most 8 d: with `size` the weighted sum of 8 d over the row's keys, every
   chunk of 16 keys adds a rounding of 2^-22 of it, and joins and the division a few.
   |error| <= size (2 e + span 2^-22 + (12 + chunks of a warp + parts) 2^-22).
Rounded to the output's type: half a step more.  lse: e + a few u of its size.  Of bf16 queries the weights are one fp16
each, every product p_j dv_j within half a step, 2^-11, of itself: sum p_j dv_j 2^-11 |code - 8| <= size 2^-11 more.

Prompts of bf16 and fp16 (tcgen05): keys and values are rounded to fp16, half a step, 2^-11: scores are off by span 2^-11 and D / 16
MMAs' 2^-22, values by 2^-11 size; weights, fp16 as well, 2^-11 size more.  Of fp16 queries keys are two exact operands, so scores
are off by 2 D / 16 MMAs' 2^-22 and a few roundings (queries by 2^-25 of their row's largest: 2^-22 span where their mean
is an eighth of it or more, as here).
"""
import numpy as np
import pytest

from oracle import attn as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q4q():
    import __graft_entry__
    __graft_entry__.build()
    import q4_quantized_matmul_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.set_device(0)
    return m


class Case:
    """A cache with sequences of `lengths` tokens, each with `rows` of queries; every byte that holds no token is 0xFF
    (scales that are NaN)."""

    def __init__(self, seed, lengths, rows, heads, kv_heads, dim, page, type="f32", garbage=0xFF, spread=1.0):
        rng = np.random.default_rng(seed)
        self.page, self.heads, self.kv_heads, self.dim, self.type = page, heads, kv_heads, dim, type
        need = [-(-n // page) for n in lengths]
        total = sum(need) + 2
        order = rng.permutation(total)
        self.pages = np.full((len(lengths), max(need + [1])), -1, np.int32)
        self.cache = np.full(total * ref.page_size(kv_heads, dim, page), garbage, np.uint8)
        at = 0
        for s, n in enumerate(lengths):
            self.pages[s, : need[s]] = order[at: at + need[s]]
            at += need[s]
            j = np.arange(n)
            if n:
                k = (rng.standard_normal((n, kv_heads, dim)) * np.exp(spread * rng.standard_normal((n, kv_heads, 1)) / 2)).astype(np.float32)
                v = (rng.standard_normal((n, kv_heads, dim)) * np.exp(spread * rng.standard_normal((n, kv_heads, 1)))).astype(np.float32)
                ref.put(self.cache, page, self.pages[s][j // page] * page + j % page, k, v)
        self.len = np.array(lengths, np.int32)
        self.first = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        q = rng.standard_normal((int(self.first[-1]), heads, dim)).astype(np.float32)
        self.q = torch.from_numpy(q).to(TYPES[type])

    def want(self, **kw):
        return ref.attend(self.q.double().numpy(), self.cache, self.page, self.kv_heads, self.pages, self.len, self.first,
                          kw.pop("scale", self.dim ** -0.5), **kw)

    def args(self):
        return (self.q.cuda(), torch.from_numpy(self.cache).cuda(), self.page, self.kv_heads, torch.from_numpy(self.pages).cuda(),
                torch.from_numpy(self.len).cuda())

    def run(self, q4q, lse=False, first=True, **kw):
        a = self.args()
        out_lse = torch.full(self.q.shape[:2], 7.0, device="cuda") if lse else None
        o = q4q.q4q_kv_attn(*a, first=torch.from_numpy(self.first).cuda() if first else None, lse=out_lse, **kw)
        return (o, out_lse) if lse else o


def on_tensor_cores(case):
    rows = case.q.shape[0] * (case.heads // case.kv_heads) / len(case.len)
    return case.type != "f32" and case.dim <= 128 and rows >= 64 and (rows >= 256 or case.q.shape[0] * case.heads * case.pages.shape[1] * case.page >= 6 << 20)


def widened(case):
    """The same, with a longer page table: few rows of prompts then take the tcgen05 kernel too."""
    more = max(0, -(-(6 << 20) // (case.q.shape[0] * case.heads * case.page)) - case.pages.shape[1])
    case.pages = np.pad(case.pages, ((0, 0), (0, more)), constant_values=-1)
    return case


def bounds(case, size, span, o):
    """(of the outputs, of lse) by the derivations above."""
    u = 2.0 ** -22
    if on_tensor_cores(case):
        e = span * ((2.0 ** -11 + case.dim // 16 * u) if case.type == "bf16" else (case.dim // 8 + 4) * u)
        tol = size * (2 * e + span * u + 2.0 ** -10 + (12 + int(case.len.max()) / 16 + 160) * u)[..., None]
        return tol + np.abs(o) * torch.finfo(TYPES[case.type]).eps / 2 + 2.0 ** -25, 2 * e + 200 * u
    e = span * (2 + 2 * (case.dim // 32 + 4)) * u
    steps = 12 + int(case.len.max()) / 16 + 160
    tol = size * (2 * e + span * u + steps * u + (2.0 ** -11 if case.type == "bf16" else 0.0))[..., None]
    eps = torch.finfo(TYPES[case.type]).eps
    return tol + np.abs(o) * eps / 2 + (0 if case.type == "f32" else 2.0 ** -25), 2 * e + steps * u


def check(case, got, lse=None, **kw):
    o, want_lse, size, span = case.want(**kw)
    tol, tol_lse = bounds(case, size, span, o)
    err = np.abs(got.double().cpu().numpy() - o)
    assert np.all(err <= tol), "off by %g of the bound at %s" % ((err / np.maximum(tol, 1e-300)).max(), np.unravel_index(np.argmax(err / np.maximum(tol, 1e-300)), err.shape))
    if lse is not None:
        got_lse = lse.double().cpu().numpy()
        seen = want_lse > -np.inf
        assert np.array_equal(got_lse == -np.inf, ~seen)
        assert np.all(np.abs(got_lse[seen] - want_lse[seen]) <= (tol_lse + 2.0 ** -22 * np.abs(want_lse))[seen])


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 100, 192, 193, 500])
def test_one_token(q4q, dim, length):
    case = Case([dim, length], [length], [1], 8, 2, dim, 16 if length % 2 else 64)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (12, 12), (10, 2), (21, 3), (16, 1), (8, 1), (40, 2)])
def test_head_layouts(q4q, type, heads, kv_heads):
    case = Case([heads, kv_heads], [70, 1, 333], [2, 1, 5], heads, kv_heads, 64, 32, type)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths,rows", [([5, 0, 40, 300], [2, 1, 0, 9]), ([33], [33]), ([257], [64]), ([3, 3], [5, 3]), ([0], [4])])
@pytest.mark.parametrize("window", [0, 1, 7, 64])
def test_ragged_rows_and_windows(q4q, type, lengths, rows, window):
    """Sequences without tokens, without rows, with fewer tokens than rows (the first rows see nothing)."""
    case = Case([len(lengths), rows[0], window], lengths, rows, 6, 3, 64, 16, type)
    got, lse = case.run(q4q, lse=True, window=window)
    check(case, got, lse, window=window)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,kv_heads,lengths,rows", [(4, 1, [40], [32]), (2, 1, [300], [150]), (1, 1, [129], [128]), (8, 2, [700], [65]),
                                                         (6, 2, [200, 1, 513], [190, 1, 300]), (3, 3, [1000, 10], [260, 10])])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_prompts(q4q, dim, heads, kv_heads, lengths, rows, window, type):
    """16-bit rows enough for the tcgen05 tiles: ragged last tiles of rows and keys, pieces cut between CTAs."""
    case = widened(Case([dim, heads, window], lengths, rows, heads, kv_heads, dim, 16 if dim == 96 else 64, type))
    assert on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True, window=window)
    check(case, got, lse, window=window)
    assert q4q.q4q_device_status() == 0
    assert torch.equal(got, case.run(q4q, window=window))


@pytest.mark.parametrize("lengths,rows", [([2048, 1126], [2048, 1126]), ([5000, 300, 2100], [1500, 300, 2100]), ([700] * 24, [333] * 24)])
@pytest.mark.parametrize("window", [0, 500])
@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_prompts_of_many_pieces(q4q, lengths, rows, window, type):
    """Every CTA has several pieces, some of a step, and shares that end with a piece near by: against the kernel of fp32 rows, which the
    other tests hold to the reference.  The bound is the derivation's with the largest of each factor: 8 d <= amax (1 + 2^-10)."""
    heads, kv_heads, dim, page = 32, 8, 64, 64
    rng = np.random.default_rng(len(lengths))
    g = torch.Generator(device="cuda").manual_seed(7)
    need = [-(-n // page) for n in lengths]
    order = torch.from_numpy(rng.permutation(sum(need)).astype(np.int32)).cuda()
    pages = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    cache = torch.full((sum(need), q4q.q4q_kv_page_size(kv_heads, dim, page)), 0xFF, dtype=torch.uint8, device="cuda")
    at, amax = 0, [0.0, 0.0]
    for s, n in enumerate(lengths):
        pages[s, : need[s]] = order[at: at + need[s]]
        at += need[s]
        k, v = (torch.randn(n, kv_heads, dim, generator=g, device="cuda") for _ in range(2))
        j = torch.arange(n, device="cuda")
        q4q.q4q_kv_append(cache, page, k, v, (pages[s].long()[j // page] * page + j % page).int())
        amax = [max(amax[0], float(k.abs().max())), max(amax[1], float(v.abs().max()))]
    first = torch.tensor([0] + rows, device="cuda").cumsum(0).int()
    q = (0.5 * torch.randn(sum(rows), heads, dim, generator=g, device="cuda")).to(TYPES[type])
    args = (cache, page, kv_heads, pages, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    want = q4q.q4q_kv_attn(q.float(), *args, first=first, window=window)
    got = q4q.q4q_kv_attn(q, *args, first=first, window=window, dst=torch.full_like(q, float("nan")))
    e = dim ** -0.5 * float(q.float().abs().sum(-1).max()) * amax[0] * (2.0 ** -11 + 2.0 ** -18)
    assert ((got.float() - want).abs() <= (2 * e + 2.0 ** -9) * amax[1] + want.abs() * 2.0 ** -8).all()
    # and closely where it counts: rounding errors are as good as independent, so far smaller over a whole head
    assert float((got.float() - want).norm() / want.norm()) < 2.0 ** -8
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_prompts_of_the_largest_values(q4q, sign):
    """All values fp16's largest: their means stay within its range."""
    case = widened(Case(34, [400], [150], 4, 2, 64, 16, "f16"))
    j = np.arange(400)
    k = np.random.default_rng(34).standard_normal((400, 2, 64)).astype(np.float32)
    ref.put(case.cache, 16, case.pages[0][j // 16] * 16 + j % 16, k, np.full_like(k, -65504.0 * sign))
    assert on_tensor_cores(case)
    got = case.run(q4q)
    assert torch.isfinite(got).all()
    check(case, got)


def test_prompts_where_rows_see_nothing(q4q):
    """More rows than tokens, sequences without tokens or rows, every row sees every key, negative and zero scales."""
    case = widened(Case(31, [100, 0, 64], [200, 180, 0], 4, 2, 64, 16, "bf16"))
    for kw in ({}, {"causal": False}, {"window": 5}, {"scale": -0.3}, {"scale": 0.0}):
        got, lse = case.run(q4q, lse=True, **kw)
        check(case, got, lse, **kw)
    assert q4q.q4q_device_status() == 0


def test_prompts_with_pages_that_are_not_there(q4q):
    case = widened(Case(32, [400, 300], [100, 120], 4, 2, 128, 16, "bf16"))
    case.pages[0, [0, 3, 24]] = -1
    case.pages[1, 7:18] = 10 ** 6
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    assert q4q.q4q_device_status() == 7


def test_prompts_rows_behind_and_strides(q4q):
    case = widened(Case(33, [160, 70], [150, 60], 4, 2, 64, 16, "bf16"))
    n = case.q.shape[0]
    wide = torch.full((n + 4, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:n, :4] = case.q.cuda()
    flat = torch.full(((n + 4) * 256 + 1,), 3.0, dtype=torch.bfloat16, device="cuda")
    q, *rest = case.args()
    for q, dst in ((wide[:, :4], torch.full((n + 4, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")), (wide[:, :4], flat[1:].view(n + 4, 4, 64))):
        lse = torch.full((n + 4, 4), 3.0, device="cuda")
        q4q.q4q_kv_attn(q, *rest, first=torch.from_numpy(case.first).cuda(), dst=dst, lse=lse)
        check(case, dst[:n], lse[:n])
        assert (dst[n:] == 3.0).all() and (lse[n:] == 3.0).all() and float(flat[0]) == 3.0


def test_every_row_sees_every_key(q4q):
    case = Case(3, [77, 9], [12, 20], 4, 2, 128, 32)
    got, lse = case.run(q4q, lse=True, causal=False)
    check(case, got, lse, causal=False)
    got = case.run(q4q, causal=False, window=10)
    check(case, got, causal=False, window=10)


@pytest.mark.parametrize("dim,lengths,rows", [(128, [4099], [1]), (128, [2000, 17, 801], [1, 1, 1]), (64, [3000, 1200], [3, 11]), (256, [1500, 700], [1, 2]),
                                              (96, [2500], [2])])
def test_cut_pieces(q4q, dim, lengths, rows):
    """More chunks than one CTA's warps take: pieces are cut between CTAs and joined."""
    case = Case([dim, len(lengths)], lengths, rows, 8, 2, dim, 64)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    assert torch.equal(got, case.run(q4q))                     # the same bits again


def test_one_row_each_without_first(q4q):
    case = Case(5, [40, 300, 9], [1, 1, 1], 8, 2, 128, 16, "bf16")
    got = case.run(q4q, first=False)
    check(case, got)
    assert torch.equal(got, case.run(q4q))


def test_scale(q4q):
    for scale in (0.0, 1.0, -0.5, 3.0):
        case = Case(6, [200], [3], 4, 2, 64, 16)
        got, lse = case.run(q4q, lse=True, scale=scale)
        check(case, got, lse, scale=scale)


@pytest.mark.parametrize("size", [2.0 ** -60, 1e-3, 300.0, 2.0 ** 40])
def test_sizes_of_queries(q4q, size):
    """The sum of |q| 8 d stays as large as elsewhere: the scale goes with the size."""
    case = Case(7, [90], [2], 4, 2, 64, 16)
    case.q = (case.q.double() * size).float()
    got = case.run(q4q, scale=0.125 / size)
    check(case, got, scale=0.125 / size)


def test_sizes_of_values_across_a_sequence(q4q):
    """Value scales from 2^-20 to 2^12 within a row's keys, the small ones weighing most."""
    rng = np.random.default_rng(8)
    case = Case(8, [640], [2], 2, 1, 64, 64)
    v = rng.standard_normal((640, 1, 64)).astype(np.float32) * (2.0 ** rng.integers(-20, 13, (640, 1, 1))).astype(np.float32)
    k = rng.standard_normal((640, 1, 64)).astype(np.float32) * 3
    j = np.arange(640)
    ref.put(case.cache, 64, case.pages[0][j // 64] * 64 + j % 64, k, v)
    got = case.run(q4q)
    check(case, got)


def test_large_scores(q4q):
    """Scores in the thousands: one key takes all."""
    case = Case(9, [300], [2], 4, 2, 128, 16)
    got = case.run(q4q, scale=100.0)
    o, _, size, span = case.want(scale=100.0)
    # the scores' errors decide between near keys: rows whose best key leads by more than they can be off by
    assert np.isfinite(got.cpu().numpy()).all()
    u, clear = 2.0 ** -22, 0
    for i in range(2):
        for h in range(4):
            k = ref.get(case.cache, 16, 2, 128, case.pages[0][np.arange(300 - 1 + i) // 16] * 16 + np.arange(300 - 1 + i) % 16)[0][:, h // 2]
            s = np.sort(100.0 * (k @ case.q[i, h].double().numpy()))
            if s[-1] - s[-2] > 30 + 2 * span[i, h] * 18 * u:
                clear += 1
                assert np.all(np.abs(got[i, h].double().cpu().numpy() - o[i, h]) <= size[i, h] * 2.0 ** -19)
    assert clear > 0


@pytest.mark.parametrize("rows,type", [(1, "f32"), (20, "f32"), (20, "bf16"), (70, "bf16")])
def test_nan_in_keys_that_a_row_does_not_see(q4q, rows, type):
    """A NaN or infinite scale of a later token, of a token before the window: rows that do not see it are
    what they are without it; rows that do are not finite in the block's dims (values) or everywhere (keys)."""
    n, window = 200, 30
    case = widened(Case(10, [n], [rows], 4, 2, 64, 16, type))
    clean = case.run(q4q, window=window).cpu()
    o, _, size, span = case.want(window=window)
    tol = torch.from_numpy(2 * bounds(case, size, span, o)[0])
    at_s = ref.places(64)[2]
    for token, of_v in ((n - 1, True), (n - 1, False), (n - rows - window - 5, True), (n - rows - window - 5, False)):
        if token < 0:
            continue
        case2 = widened(Case(10, [n], [rows], 4, 2, 64, 16, type))
        slot = int(case2.pages[0][token // 16]) * 16 + token % 16
        where = ref.chunk_of(slot, 1, 2, 64, 16) + at_s(slot % 16, of_v)[1]
        case2.cache[where: where + 2] = np.array([np.inf if token % 2 else np.nan], np.float16).view(np.uint8)
        got = case2.run(q4q, window=window).cpu()
        sees = torch.tensor([token <= n - rows + i and token > n - rows + i - window for i in range(rows)])
        assert ((got - clean).abs() <= tol)[~sees].all()
        assert ((got - clean).abs() <= tol)[:, :2].all()        # the other head
        if sees.any():
            hit = got[sees][:, 2:]
            # an infinite scale of a key times a negative sum is a score of -inf, a weight of 0: only a NaN has to show
            if of_v or token % 2 == 0:
                assert not torch.isfinite(hit[..., 32:]).all(-1).any()
            if of_v:
                assert ((hit - clean[sees][:, 2:]).abs() <= tol[sees][:, 2:])[..., :32].all()


def test_rows_behind_the_last_sequence_and_strided_queries(q4q):
    case = Case(11, [60, 70], [2, 3], 4, 2, 64, 16, "bf16")
    n = case.q.shape[0]
    wide = torch.full((n + 4, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:n, :4] = case.q.cuda()
    dst = torch.full((n + 4, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 4, 4), 3.0, device="cuda")
    q, *rest = case.args()
    got = q4q.q4q_kv_attn(wide[:, :4], *rest, first=torch.from_numpy(case.first).cuda(), dst=dst, lse=lse)
    assert got.data_ptr() == dst.data_ptr()
    check(case, dst[:n], lse[:n])
    assert (dst[n:] == 3.0).all() and (lse[n:] == 3.0).all()
    # values that are 2 bytes off a vector's alignment, in and out
    flat = torch.full((n * 8 * 64 + 1,), 5.0, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:].view(n, 8, 64)
    odd[:, :4] = case.q.cuda()
    buf = torch.full((n * 4 * 64 + 1,), 5.0, dtype=torch.bfloat16, device="cuda")
    got2 = q4q.q4q_kv_attn(odd[:, :4], *rest, first=torch.from_numpy(case.first).cuda(), dst=buf[1:].view(n, 4, 64))
    assert torch.equal(got2, dst[:n]) and float(buf[0]) == 5.0


def test_pages_that_are_not_there(q4q):
    """A page outside the cache, before or behind it, holds nothing that a row sees, and is reported."""
    for bad in (-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1):
        case = Case(12, [400, 50], [2, 1], 4, 2, 128, 16)
        case.pages[0, [0, 3, 24]] = bad
        case.pages[0, 7:13] = bad
        got, lse = case.run(q4q, lse=True)
        check(case, got, lse)
        assert q4q.q4q_device_status() == 7 and q4q.q4q_device_status() == 0
    case.pages[:] = -1
    got, lse = case.run(q4q, lse=True)
    assert (got == 0).all() and (lse == -np.inf).all() and q4q.q4q_device_status() == 7


def test_lengths_that_cannot_be(q4q):
    """More tokens than the pages hold count as those; fewer than none as none."""
    case = Case(13, [64, 32], [1, 1], 4, 2, 64, 16)
    want = case.run(q4q)
    long = Case(13, [64, 32], [1, 1], 4, 2, 64, 16)
    long.len[0] = 10 ** 9
    assert torch.equal(long.run(q4q), want) and q4q.q4q_device_status() == 7
    long.len[0] = -5
    got = long.run(q4q)
    assert (got[0] == 0).all() and torch.equal(got[1], want[1]) and q4q.q4q_device_status() == 7


def test_firsts_that_cannot_be(q4q):
    """Rows outside q are not touched, whatever first says."""
    case = Case(14, [64, 32, 20], [2, 1, 1], 4, 2, 64, 16)
    q, *rest = case.args()
    dst = torch.full((8, 4, 64), 3.0, device="cuda")
    for first in ([-7, 2, 10 ** 9, 10 ** 9], [3, 1, 0, 2 ** 31 - 1], [0, -1, -1, -1]):
        q4q.q4q_kv_attn(q, *rest, first=torch.tensor(first, dtype=torch.int32, device="cuda"), dst=dst)
        torch.cuda.synchronize()
        assert (dst[4:] == 3.0).all()
    assert q4q.q4q_device_status() == 0


def test_many_sequences(q4q):
    """More sequences than a CTA has threads, most of them short, some without rows."""
    rng = np.random.default_rng(15)
    lengths = [int(x) for x in rng.integers(0, 40, 700)]
    lengths[350] = 900
    rows = [int(x) for x in rng.integers(0, 3, 700)]
    case = Case(15, lengths, rows, 2, 1, 64, 16)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)


def test_offsets_past_32_bits(q4q):
    """A cache of 5.6 GB: the pages of a sequence lie on either side of 2^32 bytes."""
    page, heads, dim = 256, 8, 128
    size = ref.page_size(heads, dim, page)
    n = 9500
    small = Case(16, [700], [2], 16, 8, 128, page)
    cache = torch.empty(n * size, dtype=torch.uint8, device="cuda")
    at = [9499, 3, 7300]
    for i, p in enumerate(at):
        old = int(small.pages[0, i])
        cache[p * size: (p + 1) * size] = torch.from_numpy(small.cache[old * size: (old + 1) * size]).cuda()
    pages = torch.tensor([at], dtype=torch.int32, device="cuda")
    q, _, _, _, _, length = small.args()
    got = q4q.q4q_kv_attn(q, cache, page, heads, pages, length, first=torch.from_numpy(small.first).cuda())
    assert torch.equal(got, small.run(q4q))
    slots = torch.tensor([9499 * page + 5, 3 * page + 255, 7300 * page], dtype=torch.int32, device="cuda")
    k, v = q4q.q4q_kv_get_rows(cache, page, heads, dim, slots)
    old = [int(small.pages[0, 0]) * page + 5, int(small.pages[0, 1]) * page + 255, int(small.pages[0, 2]) * page]
    want = ref.get(small.cache, page, heads, dim, old)
    assert np.array_equal(k.double().cpu().numpy(), want[0]) and np.array_equal(v.double().cpu().numpy(), want[1])
    x = torch.randn(3, heads, dim, device="cuda")
    q4q.q4q_kv_append(cache, page, x, 2 * x, slots)
    again, _ = q4q.q4q_kv_get_rows(cache, page, heads, dim, slots)
    codes, d = ref.q4(x.cpu().numpy())
    assert np.array_equal(again.double().cpu().numpy(), ((codes.astype(np.float64) - 8) * d.astype(np.float64)[..., None]).reshape(3, heads, dim))


def test_timeout_path(q4q):
    case = Case(17, [500], [1], 8, 2, 128, 16)
    q4q.q4q_debug_kv_attn_timeout(*case.args(), 2_000_000)
    assert q4q.q4q_device_status() == 6 and q4q.q4q_device_status() == 0
    check(case, case.run(q4q))
    case = widened(Case(17, [500], [150], 8, 2, 64, 16, "bf16"))
    first = torch.from_numpy(case.first).cuda()
    q4q.q4q_debug_kv_attn_timeout(*case.args(), 2_000_000, first=first, path=1)
    assert q4q.q4q_device_status() == 6 and q4q.q4q_device_status() == 0
    check(case, case.run(q4q))
    with pytest.raises(q4q.Q4QError):
        q4q.q4q_debug_kv_attn_timeout(*Case(17, [500], [150], 8, 2, 64, 16).args(), 2_000_000, first=first, path=1)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 9])
def test_every_kernel_of_warp_level_mmas(q4q, dim, type, rows):
    """Each head size, type and number of column groups, with more chunks than a CTA takes."""
    case = Case([dim, rows], [300, 40, 17], [rows, 1, rows], 6, 2, dim, 32, type)
    assert not on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)


def test_streams_graphs_and_workspaces(q4q):
    """On another stream, with a workspace of the caller's, in a graph that is replayed on new contents."""
    case, other = Case(18, [600, 90], [1, 1], 8, 2, 128, 16), Case(19, [600, 90], [1, 1], 8, 2, 128, 16)
    want, want2 = case.run(q4q), other.run(q4q)
    q, cache, page, kv, pages, length = case.args()
    first = torch.from_numpy(case.first).cuda()
    ws = torch.full((q4q.q4q_kv_attn_workspace_size(2, 8, 2, 128, 2),), 0xFF, dtype=torch.uint8, device="cuda")
    dst = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q4q.q4q_kv_attn(q, cache, page, kv, pages, length, first=first, stream=side, workspace=ws)
    torch.cuda.synchronize()                             # nothing else orders the comparison behind the other stream
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4q.q4q_kv_attn(q, cache, page, kv, pages, length, first=first, dst=dst, workspace=ws)
        q4q.q4q_kv_attn(q, cache, page, kv, pages, length, first=first, dst=dst, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dst, want)
    q2, cache2, _, _, pages2, _ = other.args()
    q.copy_(q2), cache.copy_(cache2), pages.copy_(pages2)
    ws.fill_(0x7F)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dst, want2)


def test_streams_and_graphs_of_prompts(q4q):
    case, other = (widened(Case(s, [300, 150], [200, 150], 4, 2, 64, 16, "bf16")) for s in (41, 42))
    want, want2 = case.run(q4q), other.run(q4q)
    q, cache, page, kv, pages, length = case.args()
    first = torch.from_numpy(case.first).cuda()
    ws = torch.full((q4q.q4q_kv_attn_workspace_size(350, 4, 2, 64, 2, torch.bfloat16),), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q4q.q4q_kv_attn(q, cache, page, kv, pages, length, first=first, stream=side, workspace=ws)
    torch.cuda.synchronize()                             # nothing else orders the comparison behind the other stream
    assert torch.equal(got, want)
    dst, graph = torch.empty_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            q4q.q4q_kv_attn(q, cache, page, kv, pages, length, first=first, dst=dst, workspace=ws)
    q2, cache2, _, _, pages2, _ = other.args()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dst, want)
    q.copy_(q2), cache.copy_(cache2), pages.copy_(pages2), ws.fill_(0x7F)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dst, want2)
    # two calls at once, on streams and workspaces of their own
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([q4q.q4q_kv_attn(q, cache, page, kv, pages, length, first=first) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want2) for out in outs for o in out)


def test_prompts_of_many_sequences(q4q):
    """More sequences than warps share their tiles between."""
    rng = np.random.default_rng(43)
    lengths = [int(x) for x in rng.integers(0, 60, 230)]
    lengths[100] = 700
    rows = [min(int(x), n) if n else 2 for x, n in zip(rng.integers(0, 50, 230), lengths)]
    rows[100] = 600
    case = widened(Case(43, lengths, rows, 4, 1, 64, 16, "bf16"))
    assert on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("rows,type", [(1, "f32"), (3, "f16"), (9, "bf16"), (80, "bf16"), (80, "f16")])
def test_rows_of_nan_and_keys_of_nan(q4q, rows, type):
    """A row whose query is NaN is NaN, and the others are right; so is every row where all keys are NaN."""
    case, case2 = (widened(Case([44, rows], [200, 90], [rows, rows], 4, 2, 64, 16, type)) for _ in range(2))
    want = case.run(q4q)
    case.q[0, 1, 3] = float("nan")
    got, lse = case.run(q4q, lse=True)
    assert torch.isnan(got[0, 1]).all() and torch.isnan(lse[0, 1])
    # a tile's rows move their references together, so the others may round differently
    o, true_lse, size, span = case2.want()
    tol, tol_lse = bounds(case2, size, span, o)
    keep = np.ones(got.shape[:2], bool)
    keep[0, 1] = False
    assert np.all((np.abs(got.double().cpu().numpy() - o) <= tol)[keep])
    assert np.all((np.abs(lse.double().cpu().numpy() - true_lse) <= tol_lse + 2.0 ** -22 * np.abs(true_lse))[keep])
    case = widened(Case([44, rows], [200, 90], [rows, rows], 4, 2, 64, 16, type))
    k = np.full((200, 2, 64), np.nan, np.float32)
    k[:, 1] = 1.0
    j = np.arange(200)
    ref.put(case.cache, 16, case.pages[0][j // 16] * 16 + j % 16, k, np.ones_like(k))
    got, lse = case.run(q4q, lse=True)
    assert torch.isnan(got[:rows, :2]).all() and torch.isnan(lse[:rows, :2]).all()
    assert torch.isfinite(got[:rows, 2:]).all() and torch.equal(got[rows:], want[rows:])


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_two_groups_of_columns(q4q, type, dim):
    """More rows than a group holds and steps enough for two groups: by the tables' keys, most of which are not used."""
    case = Case([dim, 47], [700, 90, 33, 5], [9, 12, 10, 5], 4, 2, dim, 16, type)
    case.pages = np.pad(case.pages, ((0, 0), (0, 65536 // 16 - case.pages.shape[1])), constant_values=-1)
    assert not on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    assert torch.equal(got, case.run(q4q)) and q4q.q4q_device_status() == 0


@pytest.mark.parametrize("rows,type", [(3, "f32"), (80, "bf16")])
def test_windows_past_every_key(q4q, rows, type):
    case = widened(Case(45, [300], [rows], 4, 2, 64, 16, type))
    want = case.run(q4q)
    for window in (300, 2 ** 31, 2 ** 63 - 1):
        assert torch.equal(case.run(q4q, window=window), want)


def test_steps_with_projections(q4q):
    """As a model runs them: fused projection, norm and rotation, append, attention, output projection; prompts of two sequences, then
    single tokens in a graph whose positions, slots and lengths move on.  Every step against the references, from its own inputs."""
    import oracle
    rng = np.random.default_rng(46)
    heads, kv, dim, page, width, eps = 6, 2, 64, 16, 384, 1e-5
    rows = (heads + 2 * kv) * dim
    w_in = oracle.quantize_q4_0(rng.standard_normal((rows, width)).astype(np.float32) / 20)
    w_out = oracle.quantize_q4_0(rng.standard_normal((width, heads * dim)).astype(np.float32) / 20)
    wq, wk = ((1 + rng.standard_normal(dim) / 8).astype(np.float32) for _ in range(2))
    g_in, g_out, g_wq, g_wk = (torch.from_numpy(x).cuda() for x in (w_in, w_out, wq, wk))
    table = q4q.q4q_rope_table(64, 32)
    lengths = np.array([21, 5])
    pages = np.array([[4, 0, 6], [2, 5, 1]], np.int32)
    mirror = np.zeros(8 * ref.page_size(kv, dim, page), np.uint8)
    cache = torch.zeros(mirror.size, dtype=torch.uint8, device="cuda")
    g_pages = torch.from_numpy(pages).cuda()

    def block(x, pos, slots, kv_len, first):
        qkv = q4q.q4q_mul_mat(g_in, width, rows, x).view(-1, heads + 2 * kv, dim)
        q, _ = q4q.q4q_qk_norm_rope(qkv[:, :heads], None, g_wq, None, eps, table, pos)
        q4q.q4q_kv_append(cache, page, qkv[:, heads: heads + kv], qkv[:, heads + kv:], slots, g_wk, eps, table, pos)
        o = q4q.q4q_kv_attn(q, cache, page, kv, g_pages, kv_len, first=first)
        return qkv, q, o, q4q.q4q_mul_mat(g_out, heads * dim, width, o.view(-1, heads * dim))

    def verify(x, pos, slots, kv_len, first, got):
        qkv, q, o, y = (t.cpu().numpy() for t in got)
        want, size = oracle.mul_mat(w_in, width, rows, x)
        assert np.all(np.abs(qkv.reshape(-1, rows) - want) <= 1e-5 * size)
        t = table.cpu().numpy()
        assert np.array_equal(q, ref.norm_rope(qkv[:, :heads], wq, eps, t, pos, True).astype(np.float32))
        k = ref.norm_rope(qkv[:, heads: heads + kv], wk, eps, t, pos, True).astype(np.float32)
        ref.put(mirror, page, slots, k, qkv[:, heads + kv:])
        assert np.array_equal(cache.cpu().numpy(), mirror)
        want, _, size, span = ref.attend(q, mirror, page, kv, pages, kv_len, first, dim ** -0.5)
        u = 2.0 ** -22
        e = span * (2 + 2 * (dim // 32 + 4)) * u
        assert np.all(np.abs(o - want) <= size * (2 * e + span * u + (12 + 160 + 2) * u)[..., None] + np.abs(want) * 2.0 ** -24)
        want, size = oracle.mul_mat(w_out, heads * dim, width, o.reshape(-1, heads * dim))
        assert np.all(np.abs(y - want) <= 1e-5 * size)

    def inputs(rows_of, base):
        pos = np.concatenate([np.arange(b, b + n) for b, n in zip(base, rows_of)]).astype(np.int32)
        seq = np.repeat(np.arange(2), rows_of)
        x = rng.standard_normal((pos.size, width)).astype(np.float32)
        return x, pos, (pages[seq, pos // page] * page + pos % page).astype(np.int32), (base + rows_of).astype(np.int32), \
            np.concatenate([[0], np.cumsum(rows_of)]).astype(np.int32)

    step = inputs(lengths, np.zeros(2, np.int64))
    verify(*step, block(*(torch.from_numpy(a).cuda() for a in step)))
    one = np.ones(2, np.int64)
    held = [torch.from_numpy(a).cuda() for a in inputs(one, lengths)]
    saved = cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(*held)
    torch.cuda.synchronize()
    cache.copy_(saved)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(*held)
    for n in range(4):
        step = inputs(one, lengths + n)
        for t, a in zip(held, step):
            t.copy_(torch.from_numpy(a))
        graph.replay()
        torch.cuda.synchronize()
        verify(*step, got)
    assert q4q.q4q_device_status() == 0


def test_refusals(q4q):
    case = Case(20, [40], [1], 8, 2, 64, 16)
    q, cache, page, kv, pages, length = case.args()
    ok = dict(first=None)
    call = q4q.q4q_kv_attn
    for error, args in (
            (TypeError, (q.cpu(), cache, page, kv, pages, length)),
            (TypeError, (q.int(), cache, page, kv, pages, length)),
            (TypeError, (q, cache, page, kv, pages.long(), length)),
            (TypeError, (q, cache, page, kv, pages, length.float())),
            (ValueError, (q[0], cache, page, kv, pages, length)),
            (ValueError, (q, cache[:-1], page, kv, pages, length)),
            (ValueError, (q.transpose(1, 2), cache, page, kv, pages, length)),
            (ValueError, (q, cache, page, kv, pages[0], length)),
            (ValueError, (q, cache, page, kv, pages, length[:0])),
            (q4q.Q4QError, (q, cache, 24, kv, pages, length)),
            (q4q.Q4QError, (q, cache[:6912], page, 3, pages, length)),
            (q4q.Q4QError, (q, cache, page, 0, pages, length)),
            (q4q.Q4QError, (q[..., :32].contiguous(), cache, page, kv, pages, length))):
        with pytest.raises(error):
            call(*args, **ok)
    with pytest.raises(q4q.Q4QError):
        call(q, cache, page, kv, pages, length, window=-1)
    with pytest.raises(q4q.Q4QError):
        call(q, cache, page, kv, pages, length, scale=float("nan"))
    with pytest.raises(q4q.Q4QError):
        call(q, cache, page, kv, pages, length, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        call(q, cache, page, kv, pages, length, dst=torch.empty_like(q, dtype=torch.float16))
    with pytest.raises(ValueError):
        call(q, cache, page, kv, pages, length, dst=torch.empty_like(q)[:, :4].contiguous())
    with pytest.raises(ValueError):
        call(q, cache, page, kv, pages, length, lse=torch.empty(3, device="cuda"))
    empty = call(q[:0], cache, page, kv, pages[:0], length[:0])
    assert empty.shape == (0, 8, 64) and q4q.q4q_device_status() == 0
