"""Attention over the cache: workspaces, and cases that take much memory."""
import numpy as np
import pytest

from attn_close import EPS, assert_close
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


def close(case, got, lse, **kw):
    assert_close(case.type, case.first, got.double().cpu().numpy(), lse.double().cpu().numpy(), *case.want(**kw))


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("type", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,lengths,rows", [(4, 1, [40], [32]), (8, 2, [700], [65]), (6, 2, [200, 1, 513], [190, 1, 300]), (3, 3, [1000, 10], [260, 10]),
                                                         (2, 1, [300], [150])])
@pytest.mark.parametrize("window", [0, 20, 100])
def test_prompts_are_close(q4q, dim, type, heads, kv_heads, lengths, rows, window):
    """Within limits that reject what test_attn_close.py plants: masks that are off by one, scales by 3%, rows of another head or dim."""
    case = widened(Case([dim, heads, window, len(rows)], lengths, rows, heads, kv_heads, dim, 16 if dim == 96 else 64, type))
    assert on_tensor_cores(case)
    got, lse = case.run(q4q, lse=True, window=window)
    close(case, got, lse, window=window)
    assert torch.equal(got, case.run(q4q, window=window)) and q4q.q4q_device_status() == 0


@pytest.mark.parametrize("dim", [96, 128])
@pytest.mark.parametrize("type", ["f16", "bf16"])
@pytest.mark.parametrize("lengths,rows,window", [([2048, 1126], [2048, 1126], 0), ([5000, 300, 2100], [1500, 300, 2100], 500), ([700] * 24, [333] * 24, 0)])
def test_prompts_of_many_pieces_of_larger_heads(q4q, dim, type, lengths, rows, window):
    """Every CTA has several pieces, one stage of keys: against the kernel of fp32 rows, whose errors are 2^-10 of these; each head of each
    sequence within the limits of attn_close."""
    heads, kv_heads, page = 16, 4, 64
    g = torch.Generator(device="cuda").manual_seed(dim)
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(need), generator=g, device="cuda").int()
    pages = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    cache = torch.full((sum(need), q4q.q4q_kv_page_size(kv_heads, dim, page)), 0xFF, dtype=torch.uint8, device="cuda")
    at = 0
    for s, n in enumerate(lengths):
        pages[s, : need[s]] = order[at: at + need[s]]
        at += need[s]
        j = torch.arange(n, device="cuda")
        q4q.q4q_kv_append(cache, page, *(torch.randn(n, kv_heads, dim, generator=g, device="cuda") for _ in range(2)),
                          (pages[s].long()[j // page] * page + j % page).int())
    first = torch.tensor([0] + rows, device="cuda").cumsum(0).int()
    q = torch.randn(sum(rows), heads, dim, generator=g, device="cuda").to(TYPES[type])
    args = (cache, page, kv_heads, pages, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    lse, want_lse = (torch.empty(sum(rows), heads, device="cuda") for _ in range(2))
    want = q4q.q4q_kv_attn(q.float(), *args, first=first, window=window, lse=want_lse).double()
    got = q4q.q4q_kv_attn(q, *args, first=first, window=window, lse=lse, dst=torch.full_like(q, float("nan"))).double()
    a = 0
    for n in rows:
        o, e = want[a: a + n], got[a: a + n] - want[a: a + n]
        assert float((e.norm(dim=(0, 2)) / o.norm(dim=(0, 2))).max()) <= EPS[type]
        x, y = (lse - want_lse).double()[a: a + n], want_lse[a: a + n].abs().amax(0)
        assert bool((x.square().mean(0).sqrt() <= (dim // 8 + 4) * 2.0 ** -22 * y + 2.0 ** -17).all())
        a += n
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,lengths,rows,window", [(4, 2, [300], [200], 0), (8, 1, [150, 40], [130, 40], 0), (2, 2, [500, 257], [100, 257], 60)])
def test_prompts_with_heads_of_256(q4q, type, heads, kv_heads, lengths, rows, window):
    case = Case([256, heads, window], lengths, rows, heads, kv_heads, 256, 32, type)
    for pages in (case.pages, np.pad(case.pages, ((0, 0), (0, 65536 // 32 - case.pages.shape[1])), constant_values=-1)):
        case.pages = pages                               # few steps by the table, one group of columns; many, two
        got, lse = case.run(q4q, lse=True, window=window)
        check(case, got, lse, window=window)
        if type != "f32":
            close(case, got, lse, window=window)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_prompts_with_offsets_past_32_bits(q4q, type):
    """A cache of 5.6 GB: the pages of a sequence lie on either side of 2^32 bytes."""
    page, heads, dim = 256, 8, 128
    size, n = ref.page_size(heads, dim, page), 9500
    small = widened(Case(16, [700], [200], 16, 8, 128, page, type))
    assert on_tensor_cores(small)
    want = small.run(q4q)
    close(small, *small.run(q4q, lse=True))
    cache = torch.empty(n * size, dtype=torch.uint8, device="cuda")
    at = [9499, 3, 7300]
    q, _, _, _, pages, length = small.args()
    for i, p in enumerate(at):
        old = int(small.pages[0, i])
        cache[p * size: (p + 1) * size] = torch.from_numpy(small.cache[old * size: (old + 1) * size]).cuda()
        pages[0, i] = p
    got = q4q.q4q_kv_attn(q, cache, page, heads, pages, length, first=torch.from_numpy(small.first).cuda())
    assert torch.equal(got, want) and q4q.q4q_device_status() == 0


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths,rows", [([3000], [1]), ([2000, 700, 50], [9, 12, 3]), ([900, 400], [300, 150])])
def test_nothing_is_written_beside_results_and_workspace(q4q, dim, type, lengths, rows):
    """Workspaces of the exact size, whatever they first hold, results and lse between guards."""
    case = Case([dim, len(rows)], lengths, rows, 4, 2, dim, 16, type)
    need = q4q.q4q_kv_attn_workspace_size(sum(rows), 4, 2, dim, len(rows), TYPES[type])
    want, want_lse = case.run(q4q, lse=True)
    check(case, want, want_lse)
    guard, n = 1 << 16, want.numel()
    a = case.args()
    for fill in (0xFF, 0x00, 0x7F):
        ws = torch.full((need + guard + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        ws[:need] = fill
        dst = torch.full((n + 2 * guard,), 5.0, dtype=want.dtype, device="cuda")
        lse = torch.full((want_lse.numel() + 512,), 5.0, device="cuda")
        got = q4q.q4q_kv_attn(*a, first=torch.from_numpy(case.first).cuda(), workspace=ws[:need], dst=dst[guard: guard + n].view_as(want),
                              lse=lse[256:-256].view_as(want_lse))
        assert torch.equal(got, want) and torch.equal(lse[256:-256].view_as(want_lse), want_lse)
        assert (ws[need:] == 0xA5).all() and (dst[:guard] == 5).all() and (dst[guard + n:] == 5).all() and (lse[:256] == 5).all() and (lse[-256:] == 5).all()


@pytest.mark.parametrize("type", ["f16", "bf16"])
@pytest.mark.parametrize("prompt", [300, 40])
def test_a_prompt_beside_single_tokens(q4q, type, prompt):
    """One call for a prompt and decoding sequences, by either kernel (by the rows a sequence on average)."""
    rows = [1, 1, prompt, 1, 1, 1]
    case = Case([70, prompt], [400, 33, 500, 16, 129, 1], rows, 8, 2, 64, 16, type)
    for c in (case, widened(case)):
        got, lse = c.run(q4q, lse=True)
        check(c, got, lse)
        close(c, got, lse)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,lengths,rows", [(1024, 1, [100, 3], [1, 2]), (1024, 1024, [40], [1]), (768, 3, [70, 30], [2, 1])])
def test_the_most_heads(q4q, type, heads, kv_heads, lengths, rows):
    case = Case([heads, kv_heads], lengths, rows, heads, kv_heads, 64, 16, type)
    for c in (case, widened(case) if type != "f32" else case):
        got, lse = c.run(q4q, lse=True)
        check(c, got, lse)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
def test_the_largest_pages(q4q, type):
    case = Case(4096, [5000, 4096, 1], [1, 3, 1], 4, 2, 64, 4096, type)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    case = Case(4097, [4500], [150], 4, 2, 64, 4096, type)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 100])
def test_sequences_that_share_pages(q4q, type, rows):
    """The same prefix in every sequence's table, one page twice in one table: as many copies of it give."""
    case = Case([3, rows], [64], [rows], 4, 2, 64, 16, type)
    q, cache, page, kv, pages, length = case.args()
    table = pages.repeat(3, 1)
    table[2, 3] = table[2, 1]
    first = torch.arange(0, 3 * rows + 1, rows, dtype=torch.int32, device="cuda")
    got = q4q.q4q_kv_attn(q.repeat(3, 1, 1), cache, page, kv, table, length.repeat(3), first=first)
    again = Case([3, rows], [64], [rows], 4, 2, 64, 16, type)
    again.pages = table.cpu().numpy()
    again.len, again.first, again.q = np.full(3, 64, np.int32), first.cpu().numpy(), case.q.repeat(3, 1, 1)
    check(again, got)


@pytest.mark.parametrize("pages", [2 ** 12, 2 ** 12 + 1])
def test_tables_of_2_to_the_24_keys(q4q, pages):
    """The most that prompts take tcgen05 with, and one page more: a wait of its loaders lasts as long as a piece."""
    case = Case([24, pages], [4500, 300], [150, 90], 4, 2, 64, 4096, "bf16")
    case.pages = np.pad(case.pages, ((0, 0), (0, pages - case.pages.shape[1])), constant_values=-1)
    got, lse = case.run(q4q, lse=True)
    check(case, got, lse)
    close(case, got, lse)
    assert q4q.q4q_device_status() == 0
