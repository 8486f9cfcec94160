"""How near prompts on the tcgen05 kernel are to the 64-bit reference.

Element by element, u = 2^-22: keys are exact and queries as good as that, so a score, a sum in fp32 of D / 8 MMAs and a few roundings, is off
by e = span (D / 8 + 4) u at most; values and weights are rounded to fp16, 2^-11 each, of `size`; joins, sums of weights and the division
a few u more.  Then half a step of the result's type.
Of a sequence's head as a whole, 2-norm of the errors over that of the results: these roundings, each within half a step h (2^-11, of the result
2^-8 for bf16) and independent of the others, have a root mean square of h / sqrt(3) at most, so three of them
together no more than the largest h: the limit is twice that.  lse: partial sums of a score stay near the largest one, so each of its
D / 8 + 4 roundings is 2^-22 of that at most; 2^-18 for the sum of weights and its logarithm.
Mistakes that these limits reject: test_attn_close.py.
"""
import numpy as np

EPS = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}


def assert_close(type, first, got, got_lse, o, lse, size, span):
    """got, got_lse: of the kernel, in 64 bits; o, lse, size, span: oracle.attn.attend's."""
    dim, u = o.shape[-1], 2.0 ** -22
    e = span * (dim // 8 + 4) * u
    tol = size * (2 * e + span * u + 2.0 ** -10 + 512 * u)[..., None] + np.abs(o) * EPS[type] / 2 + 2.0 ** -25
    assert np.all(np.abs(got - o) <= tol), "%g of the elements' bound" % (np.abs(got - o) / tol).max()
    seen = lse > -np.inf
    assert np.array_equal(got_lse == -np.inf, ~seen)
    for a, b in zip(first[:-1], first[1:]):
        for h in range(o.shape[1]):
            s = seen[a:b, h]
            if not s.any():
                assert not got[a:b, h].any()
                continue
            err = np.linalg.norm(got[a:b, h] - o[a:b, h]) / np.linalg.norm(o[a:b, h])
            assert err <= EPS[type], "rows %d to %d, head %d: results off by %g" % (a, b, h, err)
            x = (got_lse - lse)[a:b, h][s]
            limit = (dim // 8 + 4) * u * np.abs(lse[a:b, h][s]).max() + 2.0 ** -18
            assert np.sqrt((x * x).mean()) <= limit, "rows %d to %d, head %d: lse off by %g" % (a, b, h, np.sqrt((x * x).mean()))
