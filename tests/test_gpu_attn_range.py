"""Attention over the cache where weights or values of a row's keys lie far apart, against oracle/attn.py (64 bits).

The bounds are those of test_gpu_attn.  Where outputs are means of many values of either sign, a bound by the sum of their sizes is loose; there the
2-norm of a whole head's error is held to its result's.  Rounding errors of weights, values and results are independent, each
within half a step, h = 2^-11 of fp16 or 2^-8 of bf16, uniform in it, so of root mean square h / sqrt(3) at most; the sum of
three of them (weights, values, result) is below sqrt(3) max(h) / sqrt(3): the limit is 2 h of the results' type.  lse is as
good as the scores, which are sums in fp32 of exact products: D / 8 + 4 roundings or cuts, 2^-22 of what has been summed, which stays near
the largest score.
"""
import numpy as np
import pytest

from oracle import attn as ref
from test_gpu_attn import Case, TYPES, check, on_tensor_cores, q4q, widened  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def put(case, s, k, v):
    j = np.arange(len(k))
    ref.put(case.cache, case.page, case.pages[s][j // case.page] * case.page + j % case.page, k.astype(np.float32), v.astype(np.float32))


def with_sink(seed, n, rows, heads, kv_heads, dim, type, nats):
    """The first key weighs exp(nats) times as much as the others do at a score of zero, and its value is zero."""
    case = Case(seed, [n], [rows], heads, kv_heads, dim, 16, type)
    rng = np.random.default_rng(seed)
    k, v = rng.standard_normal((n, kv_heads, dim)) / 4, rng.standard_normal((n, kv_heads, dim))
    k[:, :, 32:64] = 0
    k[0], v[0] = 0, 0
    # -1 in block 1 of each query: a key of -c there, which is a code of its own, scores 32 c / sqrt(D)
    k[0, :, 32:64] = -np.float16(nats * dim ** 0.5 / 32)
    put(case, 0, k, v)
    case.q[:, :, 32:64] = -1
    return case


def norm_error(got, want):
    """Of each head: the error's 2-norm over the result's."""
    e = got.double().cpu().numpy() - want
    return np.sqrt((e * e).sum((0, 2)) / (want * want).sum((0, 2)))


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_prompts_whose_first_key_outweighs_the_rest(q4q, dim, type):
    """By 2^20: weights of the rest are still normal numbers in fp16."""
    case = widened(with_sink(dim, 500, 200, 4, 2, dim, type, 20 * np.log(2)))
    assert on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    # the first row sees 301 keys
    assert norm_error(got, case.want()[0]).max() <= torch.finfo(TYPES[type]).eps
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_prompts_whose_first_key_outweighs_4096_others(q4q, type):
    """By 2^26, each of the others' values 1: their share of 2^-14 is the result.  As many sequences, all of the same tokens, as leave
    most pieces whole."""
    n, seqs, rows, heads, dim, page = 4097, 38, 64, 4, 64, 64
    pages = torch.arange(-(-n // page), dtype=torch.int32, device="cuda").repeat(seqs, 1)
    cache = torch.zeros((pages.shape[1], q4q.q4q_kv_page_size(heads, dim, page)), dtype=torch.uint8, device="cuda")
    k, v = torch.zeros(n, heads, dim, device="cuda"), -torch.ones(n, heads, dim, device="cuda")
    c = float(np.float16(26 * np.log(2) / 4))                  # scores 32 c / 8
    k[0, :, 32:], v[0] = -c, 0
    q4q.q4q_kv_append(cache, page, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
    q = torch.zeros(seqs * rows, heads, dim, dtype=TYPES[type], device="cuda")
    q[..., 32:] = -1
    lse = torch.empty(seqs * rows, heads, device="cuda")
    got = q4q.q4q_kv_attn(q, cache, page, heads, pages, torch.full((seqs,), n, dtype=torch.int32, device="cuda"),
                          first=torch.arange(0, seqs * rows + 1, rows, dtype=torch.int32, device="cuda"), causal=False, lse=lse)
    share = 4096 / (4096 + np.exp(4 * c))
    # weights of 2^-26 of the first key's are within 2^-32 of it, 2^-6 of themselves
    assert float((got.double() + share).abs().max()) <= share * (2.0 ** -6 + torch.finfo(TYPES[type]).eps)
    assert float((lse.double() - (4 * c + np.log1p(4096 * np.exp(-4 * c)))).abs().max()) <= 1e-4


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_prompts_of_scores_that_spread(q4q, dim, type):
    """Scores of 20 nats' spread: their weights count as exactly as they do."""
    case = widened(Case(dim, [400], [200], 4, 2, dim, 16, type))
    rng = np.random.default_rng(dim)
    put(case, 0, 4.5 * rng.standard_normal((400, 2, dim)), rng.standard_normal((400, 2, dim)))
    case.q = 4.5 * case.q
    assert on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True)
    o, want = case.want()[:2]
    e = lse.double().cpu().numpy() - want
    assert np.sqrt((e * e).mean()) <= (dim // 8 + 4) * 2.0 ** -22 * np.abs(want).max() + 2.0 ** -18
    assert norm_error(got, o).max() <= torch.finfo(TYPES[type]).eps


# ---------------------------------------------- few rows (warp-level MMAs) --

def few(seed, n, rows, dim, type, outlier, exponent, toward):
    """Values of about 2^exponent, but for one key of +-65504; block 1 of the queries is -1 times `toward` [heads], of the keys zero
    but for the outlier's: it scores 70 nats below the others' zero where toward is 1, above where it is -1."""
    case = Case(seed, [n], [rows], 4, 2, dim, 16, type)
    rng = np.random.default_rng(seed)
    k, v = rng.standard_normal((n, 2, dim)), rng.standard_normal((n, 2, dim)) * 2.0 ** exponent
    k[:, :, 32:64] = 0
    k[outlier, :, 32:64] = 80 * dim ** 0.5 / 32
    v[outlier] = 65504 * np.sign(v[outlier])
    put(case, 0, k, v)
    case.q[:, :, 32:64] = -torch.tensor(toward, dtype=case.q.dtype)[:, None]
    return case


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("exponent", [-2, -6, -10, -16])
def test_a_large_value_without_weight(q4q, dim, type, exponent):
    """Every row sees the key, none gives it weight; the other values count as exactly as without it."""
    for rows in (1, 3, 9):
        case = few([dim, exponent + 20, rows], 300, rows, dim, type, 77, exponent, [1, 1, 1, 1])
        got, lse = case.run(q4q, lse=True)
        check(case, got, lse)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("outlier,window", [(299, 0), (298, 50), (299 - 2 - 50, 50), (299 - 2 - 49, 50)])
def test_a_large_value_that_some_rows_do_not_see(q4q, type, outlier, window):
    for toward in ([1, 1, 1, 1], [-1, -1, -1, -1], [0, 0, 0, 0]):
        case = few([outlier, window], 300, 3, 64, type, outlier, -10, toward)
        got, lse = case.run(q4q, lse=True, window=window)
        check(case, got, lse, window=window)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [2, 9])
def test_a_large_value_that_one_head_gives_all_weight(q4q, dim, type, rows):
    """Heads of one tile, of which the first has no weight for anything else and the second none for that key."""
    case = few([dim, rows], 300, rows, dim, type, 150, -12, [-1, 1, 1, -1])
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("wide", [False, True])
def test_blocks_of_values_of_different_sizes(q4q, dim, type, wide):
    """From 2^-14 to 2^12 in the blocks of a head, rising and falling along the keys as well; with one and with two groups of columns."""
    case = Case([dim, 5], [700, 90], [12, 9] if wide else [2, 1], 4, 2, dim, 16, type)
    if wide:
        case.pages = np.pad(case.pages, ((0, 0), (0, 65536 // 16 - case.pages.shape[1])), constant_values=-1)
    rng = np.random.default_rng(dim)
    for s, n in enumerate((700, 90)):
        e = np.linspace(-14, 9, dim // 32).repeat(32) * (1 if s else -1) + 3 * np.sin(np.arange(n) / 20)[:, None, None]
        put(case, s, rng.standard_normal((n, 2, dim)), rng.standard_normal((n, 2, dim)) * 2.0 ** e)
    assert not on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    assert torch.equal(got, case.run(q4q)) and q4q.q4q_device_status() == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nats", [12, 60])
@pytest.mark.parametrize("at", [0, 400])
def test_a_key_without_value_that_outweighs_the_rest(q4q, dim, type, nats, at):
    """First or in the middle; by exp(60) the rest is what is left of the result all the same."""
    case = with_sink([dim, nats], 700, 3, 4, 2, dim, type, nats)
    if at:
        k, v = (x[:, :, :] for x in ref.get(case.cache, 16, 2, dim, case.pages[0][np.arange(700) // 16] * 16 + np.arange(700) % 16)[:2])
        order = np.arange(700)
        order[[0, at]] = order[[at, 0]]
        put(case, 0, k[order], v[order])
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
def test_negative_scales(q4q, type):
    """A cache that another program wrote may hold them: codes turned over (8 stays, 0 has no counterpart) are the same values."""
    case = Case(71, [300, 50], [2, 3], 4, 2, 64, 16, type)
    slots = np.concatenate([case.pages[0][np.arange(300) // 16] * 16 + np.arange(300) % 16, case.pages[1][np.arange(50) // 16] * 16 + np.arange(50) % 16])
    at_k, at_v, at_s = ref.places(64)
    for n, slot in enumerate(slots):
        for h in range(2):
            base = ref.chunk_of(int(slot), h, 2, 64, 16)
            for of_v in (False, True):
                where = base + at_s(int(slot) % 16, of_v) + 1
                case.cache[where] ^= np.where((np.arange(2) + n) % 3 == 0, 0x80, 0).astype(np.uint8)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_prompts_of_queries_with_one_large_value(q4q, dim, type):
    """2^18 times as large as the others, in a dim where keys are zero: the others count with all of their bits."""
    case = widened(Case([dim, 9], [400], [200], 4, 2, dim, 16, type))
    rng = np.random.default_rng(dim)
    k, v = 4096 * rng.standard_normal((400, 2, dim)), rng.standard_normal((400, 2, dim))
    k[:, :, :32] = 0
    put(case, 0, k, v)
    case.q = (case.q.float() * 2.0 ** -12).to(TYPES[type])
    case.q[:, :, 5] = 64
    assert on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True)
    o, want = case.want()[:2]
    e = lse.double().cpu().numpy() - want
    assert np.sqrt((e * e).mean()) <= (dim // 8 + 4) * 2.0 ** -22 * np.abs(want).max() + 2.0 ** -18
    assert norm_error(got, o).max() <= torch.finfo(TYPES[type]).eps


@pytest.mark.parametrize("dim", [64, 96, 256])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("values", [0, 1, -1])
def test_scores_that_rise_or_fall_along_the_keys(q4q, dim, type, rising, values):
    """By 200 nats: every step finds a new maximum, or none does; values of one size, of falling or of rising size, blocks of different ones."""
    case = Case([dim, rising, values + 1], [700], [3], 4, 2, dim, 16, type)
    rng = np.random.default_rng(dim)
    n = np.arange(700)[:, None, None]
    k, v = rng.standard_normal((700, 2, dim)) / 8, rng.standard_normal((700, 2, dim))
    # queries of -1 in block 1: key n scores 200 n / 700 nats (or 699 - n of them) beside the rest
    k[:, :, 32:64] = -(n if rising else 699 - n) * 200 / 700 * dim ** 0.5 / 32
    v *= 2.0 ** (values * 12 * (n - 350) / 350) * 2.0 ** np.linspace(-6, 6, dim // 32).repeat(32)
    put(case, 0, k, v)
    case.q[:, :, 32:64] = -1
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,type", [(1, "f32"), (5, "f16"), (9, "bf16"), (200, "bf16")])
def test_values_that_are_all_zero(q4q, dim, rows, type):
    """Of all keys, of all but the last, of a block: zeros, and lse as ever."""
    for kind in ("all", "but one", "block"):
        case = widened(Case([dim, rows], [300], [rows], 4, 2, dim, 16, type)) if rows > 99 else Case([dim, rows], [300], [rows], 4, 2, dim, 16, type)
        rng = np.random.default_rng(dim)
        k, v = (rng.standard_normal((300, 2, dim)) for _ in range(2))
        if kind == "block":
            v[:, :, 32:64] = 0
        else:
            v[: 299 if kind == "but one" else 300] = 0
        put(case, 0, k, v)
        got, lse = case.run(q4q, lse=True)
        check(case, got, lse)
        assert kind == "but one" or not got[..., 32:64].any()


@pytest.mark.parametrize("rows,type", [(2, "f32"), (3, "f16"), (9, "bf16"), (150, "f16"), (150, "bf16")])
@pytest.mark.parametrize("most", [1e5, -1e6, 4e6])
def test_scores_of_up_to_2_to_the_22(q4q, rows, type, most):
    """Of either sign; the best key takes all where it leads by more than the scores can be off by."""
    case = Case([rows, 22], [300], [rows], 4, 2, 128, 16, type)
    if rows > 99:
        case = widened(case)
    scale = float(np.float32(most / np.abs(case.want(scale=np.sign(most))[1]).max()))
    got, lse = case.run(q4q, lse=True, scale=scale)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    o, want, size, span = case.want(scale=scale)
    assert np.abs(want).max() < 2 ** 22
    e = span * 2 * (128 // 8 + 4) * 2.0 ** -22
    assert np.all(np.abs(lse - want) <= e + 2.0 ** -22 * np.abs(want) + 1)
    k = ref.get(case.cache, 16, 2, 128, case.pages[0][np.arange(300) // 16] * 16 + np.arange(300) % 16)[0]
    clear = 0
    for i in range(rows):
        for h in range(4):
            s = np.sort(scale * (k[: 300 - rows + 1 + i, h // 2] @ case.q[i, h].double().numpy()))
            if s[-1] - s[-2] > 30 + 2 * e[i, h]:
                clear += 1
                assert np.all(np.abs(got[i, h] - o[i, h]) <= size[i, h] * 2.0 ** -10 + np.abs(o[i, h]) * torch.finfo(TYPES[type]).eps / 2)
    assert clear > 0
