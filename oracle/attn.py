"""Reference of the attention operators: numpy, 64 bits, written from the formulas of include/q4q.h."""
from __future__ import annotations

import numpy as np


def f32(x):
    """64-bit values rounded to fp32."""
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def rope_table(n_pos, rot, base=10000.0):
    angle = np.arange(n_pos, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def pairs(rot, halves):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if halves else (2 * i, 2 * i + 1)


def turn(z, table, pos, halves, rounding=f32, back=False):
    """z [tokens, heads, D] by the positions' angles."""
    z = np.array(z, np.float64)
    if table is None:
        return z
    rot = table.shape[1]
    a, b = pairs(rot, halves)
    c, s = table[pos, None, : rot // 2].astype(np.float64), table[pos, None, rot // 2:].astype(np.float64)
    s = -s if back else s
    x, y = z[..., a], z[..., b]
    z[..., a] = rounding(rounding(x * c) - rounding(y * s))
    z[..., b] = rounding(rounding(y * c) + rounding(x * s))
    return z


def inverse_norm(x, eps):
    x = np.asarray(x, np.float64)
    return f32(1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + float(np.float32(eps))))


def norm_rope(x, w, eps, table, pos, halves):
    """The fp32 values of q4q_qk_norm_rope, before their last rounding."""
    x = np.asarray(x, np.float64)
    z = x if w is None else f32(f32(x * inverse_norm(x, eps)) * np.asarray(w, np.float64))
    return turn(z, table, pos, halves)


def norm_rope_back(g, x, w, eps, table, pos, halves):
    """(dx, dw or None) in 64 bits."""
    dz = turn(g, table, pos, halves, rounding=lambda v: v, back=True)
    if w is None:
        return dz, None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + float(np.float32(eps)))
    xh, dh = x * r, dz * w
    return r * (dh - xh * np.mean(dh * xh, -1, keepdims=True)), (dz * xh).sum((0, 1))


# ------------------------------------------------------------------ cache --

def q4(x):
    """fp32 [..., D] -> codes 0 .. 15 [..., D / 32, 32] and scales fp16 [..., D / 32]."""
    b = np.asarray(x, np.float32)
    b = b.reshape(*b.shape[:-1], -1, 32)
    finite = np.isfinite(b).all(-1)
    b = np.where(finite[..., None], np.clip(b, -65504, 65504), 0).astype(np.float32)
    d = (np.abs(b).max(-1) / np.float32(8)).astype(np.float32)
    with np.errstate(all="ignore"):
        t = np.where(d[..., None] > 0, b / np.where(d > 0, d, 1)[..., None], 0).astype(np.float32).astype(np.float64)
    code = np.clip(np.sign(t) * np.floor(np.abs(t) + 0.5), -8, 7) + 8
    return code.astype(np.uint8), np.where(finite, d, np.nan).astype(np.float16)


def places(dim):
    """For each dim: byte of the chunk and shift of token i's K and V code, byte of its scales: functions of i."""
    c = np.arange(dim)
    blocks, b, r = dim // 32, c // 32, c % 32
    k = lambda i: (i * (dim // 2) + (r // 8 * blocks + b) * 4 + r % 8 // 2, r % 2 * 4)  # noqa: E731
    v = lambda i: (8 * dim + i // 8 * 4 * dim + ((r // 4 * 4 + i % 8 // 2) * blocks + b) * 4 + i % 2 * 2 + r % 4 // 2, r % 2 * 4)  # noqa: E731
    scales = lambda i, of_v: (17 if of_v else 16) * dim + (i * blocks + np.arange(blocks)) * 2  # noqa: E731
    return k, v, scales


def page_size(heads, dim, page):
    return heads * (page // 16) * 18 * dim


def chunk_of(slot, head, heads, dim, page):
    """Offset of the chunk of a slot and head."""
    return (slot // page) * page_size(heads, dim, page) + (head * (page // 16) + slot % page // 16) * 18 * dim


def put(cache, page, slots, k, v):
    """Encode k and v [tokens, heads, D] (fp32 values) into a cache, uint8 [bytes], in place."""
    heads, dim = k.shape[1:]
    at_k, at_v, at_s = places(dim)
    for x, at, of_v in ((k, at_k, False), (v, at_v, True)):
        codes, d = q4(x)
        for t, slot in enumerate(slots):
            if slot < 0 or slot >= cache.size // page_size(heads, dim, page) * page:
                continue
            for h in range(heads):
                base = chunk_of(int(slot), h, heads, dim, page)
                byte, shift = at(int(slot) % 16)
                for half in (0, 4):
                    m = shift == half
                    cache[base + byte[m]] = (cache[base + byte[m]] & (0xF0 if half == 0 else 0x0F)) | (codes[t, h].reshape(-1)[m] << half)
                where = base + at_s(int(slot) % 16, of_v)
                raw = d[t, h].view(np.uint8).reshape(-1, 2)
                cache[where], cache[where + 1] = raw[:, 0], raw[:, 1]
    return cache


def get(cache, page, heads, dim, slots):
    """(keys, values, key scales, value scales) of slots in 64 bits, scales spread over their dims."""
    at_k, at_v, at_s = places(dim)
    out = [np.zeros((len(slots), heads, dim)) for _ in range(4)]
    for t, slot in enumerate(int(s) for s in slots):
        for h in range(heads):
            base = chunk_of(slot, h, heads, dim, page)
            for n, (at, of_v) in enumerate(((at_k, False), (at_v, True))):
                byte, shift = at(slot % 16)
                where = base + at_s(slot % 16, of_v)
                d = np.stack([cache[where], cache[where + 1]], -1).reshape(-1).view(np.float16).astype(np.float64).repeat(32)
                out[2 + n][t, h] = d
                out[n][t, h] = (((cache[base + byte] >> shift) & 15).astype(np.float64) - 8) * d
    return out


# -------------------------------------------------------------- attention --

def attend(q, cache, page, kv_heads, pages, kv_len, first, scale, causal=True, window=0):
    """Outputs [rows, heads, D], lse [rows, heads], and what the bounds of a test take: `size`, the weighted sum of the
    largest values that the values' scales allow, and `span`, the largest |scale| sum |q| 8 d of a row's keys."""
    q = np.asarray(q, np.float64)
    rows, heads, dim = q.shape
    o, lse, size, span = np.zeros_like(q), np.full((rows, heads), -np.inf), np.zeros_like(q), np.zeros((rows, heads))
    for s, length in enumerate(int(n) for n in kv_len):
        r0, r1 = (s, s + 1) if first is None else (int(first[s]), int(first[s + 1]))
        if r1 <= r0 or length <= 0:
            continue
        j = np.arange(length)
        table = np.asarray(pages[s])[j // page]
        known = (table >= 0) & (table < cache.size // page_size(kv_heads, dim, page))
        k, v, kd, vd = get(cache, page, kv_heads, dim, np.where(known, table, 0) * page + j % page)
        for i in range(r0, r1):
            last = length - (r1 - r0) + (i - r0) if causal else length - 1
            seen = known & (j <= last) & ((j > last - window) if window else True)
            if not seen.any():
                continue
            for h in range(heads):
                g = h // (heads // kv_heads)
                x = scale * (k[seen, g] @ q[i, h])
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                o[i, h] = p @ v[seen, g] / l
                lse[i, h] = m + np.log(l)
                size[i, h] = p @ (8 * np.abs(vd[seen, g])) / l
                span[i, h] = (abs(scale) * (8 * np.abs(kd[seen, g])) @ np.abs(q[i, h])).max()
    return o, lse, size, span
