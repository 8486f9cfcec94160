"""Every form of the MXFP4 products on the GPU, dense and by expert, to the last bit.

The operands are whole numbers that both formats hold: weights {0, 1, 2, 3, 4, 6} and activations
{0, 1, 2, 3, 4, 6} (MXFP4) or 0 to 7 (MXFP8), signed, times 1 or 2 block by block.  A product is then a whole
number up to 7 * 6 * 4 = 168 and a sum of at most 20992 of them is below 2^22: fp32 holds every partial sum in
any order, also where terms are aligned and cut 24 bits below the largest, so results have to be equal, and a
single value that is left out, taken twice or scaled by another block's scale is seen.
"""
import numpy as np
import pytest

from mx_forms import FORMS, form, sizes
from oracle import mx
from test_gpu_experts import choices
from test_gpu_mxfp4 import q4q  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def whole(g, rows, k, values, full):
    """[rows, k] of the signed values times 1 or 2 for each block; full: 6 in every block (a scale byte of 127 or 128)."""
    v = torch.tensor(values, dtype=torch.float32, device="cuda")[torch.randint(0, len(values), (rows, k // 32, 32), generator=g, device="cuda")]
    if full:
        v[..., 5] = 6.0
    v *= torch.randint(0, 2, v.shape, generator=g, device="cuda") * 2 - 1
    v *= torch.randint(1, 3, v.shape[:2], generator=g, device="cuda")[..., None]
    return v.reshape(rows, k)


def operands(q4q, g, k, rows, tokens, matrices, acts):  # noqa: F811
    w = torch.stack([whole(g, rows, k, [0, 1, 2, 3, 4, 6], True) for _ in range(matrices)])
    packed = q4q.q4q_quantize_mxfp4(w)
    assert torch.equal(q4q.q4q_get_rows_mxfp4(packed[0], k, rows), w[0])
    x = whole(g, tokens, k, [0, 1, 2, 3, 4, 6] if acts == 0 else list(range(8)), acts == 0)
    return packed, w, x


def times(x, w):
    return (x.double() @ w.double().T).float()


def lib_and_sms():
    from q4_quantized_matmul_gb300 import _lib
    return _lib.load(), torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("acts", [0, 1])
@pytest.mark.parametrize("wanted", FORMS, ids=lambda f: "%d-%d-%d" % f)
def test_every_form_of_the_product(q4q, wanted, acts):  # noqa: F811
    lib, sms = lib_and_sms()
    k, rows, tokens, _, _ = sizes(lib, acts, False, sms)[wanted]
    g = torch.Generator(device="cuda").manual_seed(k + rows + tokens + acts)
    packed, w, x = operands(q4q, g, k, rows, tokens, 1, acts)
    assert torch.equal(q4q.q4q_mul_mat_mxfp4(packed[0], k, rows, x, acts), times(x, w[0])), (k, rows, tokens)
    # one token more or fewer, where that keeps the form
    for n in (tokens - 1, tokens + 1):
        if n > 0 and form(lib, k, rows, n, n, 0, acts, sms) == wanted:
            y = whole(g, n, k, [0, 1, 2, 3, 4, 6], True)
            assert torch.equal(q4q.q4q_mul_mat_mxfp4(packed[0], k, rows, y, acts), times(y, w[0])), (k, rows, n)
    assert q4q.q4q_device_status() == 0


@pytest.mark.parametrize("acts", [0, 1])
@pytest.mark.parametrize("wanted", FORMS, ids=lambda f: "%d-%d-%d" % f)
def test_every_form_of_the_experts_products(q4q, wanted, acts):  # noqa: F811
    lib, sms = lib_and_sms()
    k, rows, tokens, top, experts = sizes(lib, acts, True, sms)[wanted]
    g = torch.Generator(device="cuda").manual_seed(k + rows + tokens + experts + acts)
    packed, w, x = operands(q4q, g, k, rows, tokens, experts, acts)
    ids = choices(np.random.default_rng([k, rows, tokens]), tokens, top, experts)
    ids[: tokens // 3, 0] = experts - 1                       # one expert has more than its share
    first, slot, _ = mx.sort(ids, experts)
    order = q4q.q4q_moe_sort(torch.from_numpy(ids).cuda(), experts)
    got = q4q.q4q_mul_mat_id_mxfp4(packed, k, rows, x, order[0], order[1], top, acts)
    token = torch.from_numpy(slot.astype(np.int64) // top).cuda()
    for e in range(experts):
        r = slice(int(first[e]), int(first[e + 1]))
        assert torch.equal(got[r], times(x[token[r]], w[e])), (k, rows, tokens, top, experts, e)
    assert not got[int(first[experts]):].any()
    # the same rows sorted beforehand
    assert torch.equal(q4q.q4q_mul_mat_id_mxfp4(packed, k, rows, x[token], order[0], acts=acts), got)
    assert q4q.q4q_device_status() == 0
