"""MXFP4 and MXFP8 blocks, their products and the experts' rows, in plain numpy and 64 bits.

Written from the formats' definitions (32 values along K and one E8M0 scale; E2M1 or E4M3
elements), apart from the kernels: elements are rounded by comparing with the midpoints of
the format's value grid.  Test infrastructure only.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([i * 2.0 ** -9 if i < 8 else (1 + (i % 8) / 8) * 2.0 ** (i // 8 - 7) for i in range(127)])


def up(v, m):
    return (v + m - 1) // m * m


def nearest(a, grid):
    """Index into the ascending `grid` of the nearest value, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    even = np.arange(mid.size) % 2 == 0
    return np.searchsorted(mid[even], a, side="left") + np.searchsorted(mid[~even], a, side="right")


def encode(x, fmt):
    """float rows [n, K] -> (codes uint8 [n, K], scale bytes uint8 [n, K / 32], values float64 [n, K])."""
    grid, emax = (E2M1, 2) if fmt == "mxfp4" else (E4M3, 8)
    b = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - emax, -127).clip(min=-127)
    t = np.ldexp(b, -e[..., None])
    i = nearest(np.abs(t), grid)
    codes = (i | (np.signbit(t) * (8 if fmt == "mxfp4" else 128))).astype(np.uint8)
    codes[bad] = 0
    values = np.where(bad[..., None], np.nan, np.copysign(np.ldexp(grid[i], e[..., None]), t))
    return codes.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8), values.reshape(x.shape)


def pack(w):
    """float [rows, K] -> (the bytes of the MXFP4 matrix, its values float64)."""
    rows, k = w.shape
    kp = up(k, 256)
    codes, scales, values = encode(w, "mxfp4")
    full = np.zeros((rows, kp), np.uint8)
    full[:, :k] = codes
    plane = (full[:, 0::2] | (full[:, 1::2] << 4)).reshape(-1)
    out = np.zeros(up(plane.size, 256) + up(rows, 128) * kp // 32, np.uint8)
    out[:plane.size] = plane
    base = up(plane.size, 256)
    r, b = np.meshgrid(np.arange(rows), np.arange(k // 32), indexing="ij")
    out[base + (r // 128 * (kp // 128) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4] = scales
    return out, values


def sort(ids, n_experts):
    """(first, slot, row) of q4q_moe_sort, by a plain loop."""
    flat = [int(i) for i in np.asarray(ids).reshape(-1)]
    bins = [[s for s, i in enumerate(flat) if i == e] for e in range(n_experts)] if n_experts * len(flat) < 1 << 22 else None
    if bins is None:
        bins = [[] for _ in range(n_experts)]
        for s, i in enumerate(flat):
            if 0 <= i < n_experts:
                bins[i].append(s)
    slot = [s for b in bins for s in b]
    first = np.cumsum([0] + [len(b) for b in bins]).astype(np.int32)
    slot += [s for s, i in enumerate(flat) if not 0 <= i < n_experts]
    row = np.empty(len(flat), np.int32)
    row[np.array(slot, np.int64)] = np.arange(len(flat), dtype=np.int32)
    return first, np.array(slot, np.int32), row
