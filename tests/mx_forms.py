"""Sizes at which each form of the MXFP4 products is taken.

A form is (tokens of a tile, CTAs that run its MMAs, CTAs that share its K).  form() asks the library's own
choice; sizes() finds, for a device of so many SMs, the cheapest of a grid of uneven sizes for every form, so
that what the choice's constants are never takes a form out of the tests unseen.
"""
import ctypes
import functools

FORMS = [(bn, 1, split) for bn in (8, 16, 32, 64) for split in (1, 2, 4, 8)] + [(64, 2, 1), (128, 2, 1), (256, 2, 1)]

# none a multiple of a tile's 128 rows, nor of the K of a stage; tokens that do not fill their tiles among them
KS = [96, 288, 544, 1056, 1504, 2080, 4128, 7200, 14368, 20992]
ROWS = [130, 261, 520, 777, 1500, 2500, 4100, 6000, 9700, 14337, 20001]
TOKENS = [3, 7, 9, 13, 21, 30, 33, 50, 65, 100, 129, 200, 257, 300, 520, 1000]
EXPERTS = [3, 8, 20, 100]


def form(lib, k, rows, n_rows, tokens, experts, acts, sms):
    out = (ctypes.c_int * 3)()
    assert lib.q4q_debug_mxfp4_form(k, rows, n_rows, tokens, experts, acts, sms, out) == 0
    return tuple(out)


@functools.lru_cache(maxsize=None)
def sizes(lib, acts, by_expert, sms):
    """{form: (K, rows, tokens, top_k, experts)}; experts 0 and top_k 1 where not by_expert."""
    best = {}
    for experts in EXPERTS if by_expert else [0]:
        for top in (1, 2, 4) if by_expert else (1,):
            for k in KS:
                for rows in ROWS:
                    for tokens in TOKENS:
                        cost = max(experts, 1) * rows * k + 10 * tokens * top * (rows + k)
                        if cost > 4e8 or top > max(experts, 1):
                            continue
                        f = form(lib, k, rows, tokens * top, tokens, experts, acts, sms)
                        if f not in best or cost < best[f][0]:
                            best[f] = (cost, (k, rows, tokens, top, experts))
    return {f: v[1] for f, v in best.items()}
