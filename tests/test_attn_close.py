"""The limits of attn_close.py reject mistakes, planted in the reference."""
import numpy as np
import pytest

from attn_close import assert_close

torch = pytest.importorskip("torch")
from test_gpu_attn import TYPES, Case  # noqa: E402


def stored(x, type):
    return torch.from_numpy(x).to(TYPES[type]).double().numpy()


@pytest.mark.parametrize("type", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads,lengths,rows,window", [(64, 2, [300], [150], 0), (128, 8, [700], [65], 0), (96, 3, [250, 10], [130, 10], 100),
                                                           (128, 2, [300], [150], 100)])
def test_mistakes_are_rejected(type, dim, heads, lengths, rows, window):
    case = Case([dim, heads, window], lengths, rows, heads, 1, dim, 16, type)
    o, lse, size, span = case.want(window=window)

    def passes(o2, lse2):
        try:
            assert_close(type, case.first, stored(o2, type), lse2, o, lse, size, span)
        except AssertionError:
            return False
        return True
    assert passes(o, lse)
    assert not passes(np.zeros_like(o), lse)
    for wrong in (dict(window=window, scale=1.03 * dim ** -0.5), dict(window=window + 1 if window else 200), dict(window=window - 1) if window else dict(causal=False)):
        assert not passes(*case.want(**wrong)[:2]), wrong
        assert not passes(case.want(**wrong)[0], lse), wrong
        assert not passes(o, case.want(**wrong)[1]), wrong
    case.len = case.len - 1                            # every row's last key
    assert not passes(*case.want(window=window)[:2])
    case.len = case.len + 1
    case.q = case.q.flip(1)                            # another head's queries
    assert heads == 1 or not passes(*case.want(window=window)[:2])
    for wrong in (o * (1 + 2 * np.finfo(np.float32).eps * 2 ** 16), np.roll(o, 1, 0), np.roll(o, 32, 2)):
        assert not passes(wrong, lse)
