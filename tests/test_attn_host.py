"""What the attention calls refuse and compute without a GPU, and how their kernels may read memory."""
import ctypes
import os

import numpy as np
import pytest

from oracle import attn as ref
from test_dependent_launch import CSRC, NON_COHERENT, code

NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 7


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from q4_quantized_matmul_gb300 import _lib
    return _lib.load()


P = ctypes.c_void_p
AT, ODD = P(0x1000), P(0x1001)


def test_page_size(lib):
    n = ctypes.c_size_t(0)
    for heads, dim, page in ((8, 128, 64), (1, 64, 16), (12, 96, 4096), (1024, 256, 16)):
        assert lib.q4q_kv_page_size(heads, dim, page, ctypes.byref(n)) == 0 and n.value == ref.page_size(heads, dim, page)
    for heads, dim, page in ((0, 128, 64), (8, 80, 64), (8, 128, 8), (8, 128, 48), (8, 128, 8192), (1025, 64, 16), (1024, 256, 4096 * 2)):
        assert lib.q4q_kv_page_size(heads, dim, page, ctypes.byref(n)) == SHAPE
    assert lib.q4q_kv_page_size(8, 128, 64, None) == NULL


def test_norm_rope_refuses(lib):
    def call(q=AT, q_stride=256, qh=4, k=AT, k_stride=128, kh=2, type=0, dim=64, n=3, qw=AT, kw=None, eps=1e-6, table=AT, n_pos=9, rot=64, mode=1,
             pos=AT, q_dst=AT, k_dst=AT):
        return lib.q4q_qk_norm_rope(q, q_stride, qh, k, k_stride, kh, type, dim, n, qw, kw, eps, table, n_pos, rot, mode, pos, q_dst, k_dst, None)
    for want, kw in ((SHAPE, dict(dim=80)), (SHAPE, dict(q_stride=255)), (SHAPE, dict(k_stride=127)), (SHAPE, dict(qh=1025, q_stride=10 ** 6)),
                     (SHAPE, dict(kh=-1)), (SHAPE, dict(n=-1)), (SHAPE, dict(rot=72)), (SHAPE, dict(rot=80)), (SHAPE, dict(rot=0)), (SHAPE, dict(n_pos=-1)),
                     (ARG, dict(type=3)), (ARG, dict(mode=2)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("nan"))), (NULL, dict(q=None)),
                     (NULL, dict(k_dst=None)), (NULL, dict(pos=None)), (ALIGN, dict(q=ODD)), (ALIGN, dict(qw=P(0x1004))), (ALIGN, dict(table=P(0x1008))),
                     (0, dict(n=0, q=None, q_dst=None)), (0, dict(qh=0, kh=0))):
        assert call(**kw) == want, kw


def test_append_and_rows_refuse(lib):
    def append(cache=AT, pages=4, page=16, k=AT, ks=128, v=AT, vs=128, type=0, heads=2, dim=64, n=3, slots=AT, w=None, eps=0.0, table=None, n_pos=0, rot=0,
               mode=0, pos=None):
        return lib.q4q_kv_append(cache, pages, page, k, ks, v, vs, type, heads, dim, n, slots, w, eps, table, n_pos, rot, mode, pos, None)
    for want, kw in ((SHAPE, dict(page=24)), (SHAPE, dict(dim=32)), (SHAPE, dict(heads=0)), (SHAPE, dict(ks=127)), (SHAPE, dict(vs=1)), (SHAPE, dict(pages=-1)),
                     (SHAPE, dict(pages=1 << 27)), (SHAPE, dict(n=-1)), (SHAPE, dict(table=AT, rot=20, pos=AT)), (ARG, dict(type=-1)), (ARG, dict(mode=7)),
                     (NULL, dict(slots=None)), (NULL, dict(v=None)), (NULL, dict(table=AT, rot=16)), (ALIGN, dict(cache=P(0x1008))), (ALIGN, dict(k=ODD)),
                     (0, dict(n=0, cache=None))):
        assert append(**kw) == want, kw
    rows = lib.q4q_kv_get_rows
    assert rows(AT, 4, 16, 2, 64, AT, -1, AT, AT, 0, None) == SHAPE and rows(AT, 4, 16, 2, 64, AT, 3, AT, AT, 9, None) == ARG
    assert rows(AT, 4, 16, 2, 64, None, 3, AT, AT, 0, None) == NULL and rows(AT, 4, 16, 2, 64, AT, 3, ODD, AT, 0, None) == ALIGN
    assert rows(AT, 4, 16, 2, 64, AT, 3, None, None, 0, None) == 0 and rows(AT, 4, 16, 2, 64, AT, 0, AT, AT, 0, None) == 0


def test_attention_refuses(lib):
    def call(q=AT, stride=256, type=0, n_q=3, heads=4, kv=2, dim=64, cache=AT, pages=4, page=16, table=AT, most=2, len=AT, first=AT, seqs=2, scale=0.1,
             causal=1, window=0, dst=P(0x100000), lse=None, ws=AT, size=0):
        return lib.q4q_kv_attn(q, stride, type, n_q, heads, kv, dim, cache, pages, page, table, most, len, first, seqs, scale, causal, window, dst, lse, ws,
                               size, None)
    for want, kw in ((SHAPE, dict(dim=72)), (SHAPE, dict(heads=5)), (SHAPE, dict(heads=0)), (SHAPE, dict(stride=255)), (SHAPE, dict(n_q=1 << 24)),
                     (SHAPE, dict(n_q=-1)), (SHAPE, dict(seqs=1 << 20)), (SHAPE, dict(most=1 << 26)), (SHAPE, dict(window=-1)), (SHAPE, dict(page=17)),
                     (SHAPE, dict(first=None, seqs=4)), (SHAPE, dict(n_q=1 << 23, heads=512, kv=2, stride=512 * 64)), (ARG, dict(type=5)),
                     (ARG, dict(scale=float("nan"))), (NULL, dict(q=None)), (NULL, dict(dst=None)), (NULL, dict(len=None)), (NULL, dict(table=None)),
                     (NULL, dict(ws=None)), (NULL, dict(cache=None)), (ALIGN, dict(ws=P(0x1010))), (ALIGN, dict(cache=P(0x1004))), (ALIGN, dict(lse=ODD)), (ARG, dict(dst=AT)),
                     (ARG, dict(q=P(0x1000), dst=P(0x1000 + 4 * (2 * 256 + 256) - 4))), (ARG, dict(q=P(0x9000), dst=P(0x9000 - 4 * 3 * 256 + 4))),
                     (0, dict(n_q=0)), (0, dict(seqs=0))):
        assert call(**kw) == want, kw
    n = ctypes.c_size_t(0)
    assert lib.q4q_kv_attn_workspace_size(3, 4, 3, 64, 2, 0, ctypes.byref(n)) == SHAPE
    assert lib.q4q_kv_attn_workspace_size(3, 4, 2, 65, 2, 0, ctypes.byref(n)) == SHAPE
    assert lib.q4q_kv_attn_workspace_size(3, 4, 2, 64, 2, 4, ctypes.byref(n)) == ARG
    assert lib.q4q_kv_attn_workspace_size(3, 4, 2, 64, 2, 0, None) == NULL
    assert lib.q4q_rope_table(AT, 4, 24, 1e4, None) == SHAPE and lib.q4q_rope_table(AT, 4, 32, 0.0, None) == ARG and lib.q4q_rope_table(None, 0, 32, 1e4, None) == 0


def test_attention_kernels_read_coherently():
    """They start before the work ahead of them ends (see test_dependent_launch)."""
    names = [n for n in sorted(os.listdir(CSRC)) if n.startswith(("q4q_attn", "q4q_kv", "q4q_rope")) and n.endswith((".cu", ".cuh"))]
    assert {"q4q_attn_kernel.cuh", "q4q_attn_tc.cu", "q4q_kv.cu", "q4q_rope.cu", "q4q_attn.cuh"} <= set(names)
    for name in names:
        assert NON_COHERENT.findall(code(name)) == [], name


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_reference_cache(dim):
    """Every nibble and scale of a chunk belongs to one value; what is put comes back within the encoding's step."""
    k, v, scales = ref.places(dim)
    seen = np.zeros(18 * dim, np.int64)
    for i in range(16):
        for byte, shift in (k(i), v(i)):
            np.add.at(seen, byte, 1)
            assert set(shift) == {0, 4}
        for of_v in (False, True):
            at = scales(i, of_v)
            np.add.at(seen, at, 2), np.add.at(seen, at + 1, 2)
    assert (seen == 2).all()
    rng = np.random.default_rng(dim)
    x, y = (rng.standard_normal((20, 3, dim)).astype(np.float32) for _ in range(2))
    slots = rng.permutation(3 * 32)[:20]
    cache = ref.put(rng.integers(0, 256, 3 * ref.page_size(3, dim, 32)).astype(np.uint8), 32, slots, x, y)
    a, b, da, db = ref.get(cache, 32, 3, dim, slots)
    # a rounding is half a step, the largest positive value's code a whole one; the scale is rounded to fp16 (2^-11)
    assert np.all(np.abs(a - x) <= da * (1 + 2.0 ** -6)) and np.all(np.abs(b - y) <= db * (1 + 2.0 ** -6))


def test_reference_attention_is_softmax():
    """The reference on two sequences against a softmax written out."""
    rng = np.random.default_rng(0)
    cache = ref.put(np.zeros(4 * ref.page_size(1, 64, 16), np.uint8), 16, range(64), *(rng.standard_normal((64, 1, 64)).astype(np.float32) for _ in range(2)))
    q = rng.standard_normal((3, 2, 64))
    o, lse, _, _ = ref.attend(q, cache, 16, 1, [[0, 1], [3, 2]], [20, 17], [0, 2, 3], 0.125)
    slots = np.concatenate([np.arange(48, 64), [32]])
    k, v, _, _ = ref.get(cache, 16, 1, 64, slots)
    w = np.exp(0.125 * k[:, 0] @ q[2, 1])
    assert np.allclose(o[2, 1], w @ v[:, 0] / w.sum(), rtol=1e-12) and np.isclose(lse[2, 1], np.log(w.sum()))
    k, v, _, _ = ref.get(cache, 16, 1, 64, np.arange(19))
    w = np.exp(0.125 * k[:, 0] @ q[0, 0])
    assert np.allclose(o[0, 0], w @ v[:, 0] / w.sum(), rtol=1e-12)


@pytest.mark.parametrize("bits", [8, 11])
def test_ties_of_16_bit_rows(bits):
    """The encoder's way with rows of a 16-bit type: t = x rcp(d) (1 + 2^-20), rounded to nearest, gives the code that rounding the
    quotient half away from zero does, for every reciprocal within an ulp and mantissas of this many bits."""
    rng = np.random.default_rng(1)
    m = np.arange(1 << bits - 1, 1 << bits, dtype=np.float64)
    for largest in m if bits == 8 else rng.choice(m, 60, replace=False):
        d = np.float32(largest / 8)
        for e in range(0, -6, -1):
            x = m * 2.0 ** e
            x = x[x <= largest].astype(np.float32)
            want = np.minimum(np.floor((x / d).astype(np.float32).astype(np.float64) + 0.5), 7)
            for ulp in (-1, 0, 1):
                inv = np.float32((np.float32(1) / d) * (1 + ulp * 2.0 ** -23))
                inv = np.float32(np.float64(inv) + np.float64(inv) * 2.0 ** -20)
                assert np.array_equal(np.rint(np.minimum((x * inv).astype(np.float32), np.float32(7)).astype(np.float64)), want)
