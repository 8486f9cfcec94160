"""Cases of the attention operators: norms and rotation of queries and keys, the paged 4-bit cache, attention over it.

Norm and rotation of one head's row x (D values) of a token at position p:
    r = 1 / sqrt(mean(x^2) + eps) in 64 bits, rounded to fp32;  z = (x * r) * w, or z = x without a weight
    a' = a * c - b * s,  b' = b * c + a * s   for the pairs (a, b) of z's first `rot` values, (z[i], z[i + rot / 2])
or, interleaved, (z[2i], z[2i + 1]), c and s from row p of a table of cosines and sines; each product, difference and
sum is rounded to fp32.

The cache keeps Q4_0 blocks of 32 values: d = amax / 8 in fp32, code = round(x / d) (fp32 quotient, half away from
zero) limited to [-8, 7], plus 8; the value is (code - 8) * fp16(d).  A page holds `page` tokens: for each key-value
head and 16 tokens a chunk of 18 D bytes:
    K codes  [16 tokens][4 t][D / 32 blocks b] words, nibble n: dim 32 b + 8 t + n
    V codes  [2 octets][8 g][4 pairs][D / 32 blocks b] words, low half the pair's first token: nibble n: dim 32 b + 4 g + n
    K scales [16][D / 32] fp16, V scales likewise.

Attention of query i of a sequence's n (the cache holds their keys already): softmax over the keys j of
sum_d q_d K_jd / sqrt(D), j <= L - n + i, and j > L - n + i - window where there is a window; times V.
"""
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decoded token's queries and keys
        {"name": "norm_rope_1", "op": "norm_rope", "tokens": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": "halves",
         "norm": True, "train": False, "type": "f32"},
        # an odd prompt, part of each head rotated, interleaved pairs
        {"name": "norm_rope_517", "op": "norm_rope", "tokens": 517, "q_heads": 16, "kv_heads": 4, "dim": 96, "rot": 48, "pairs": "interleaved",
         "norm": True, "train": False, "type": "f16"},
        # a training batch, forward and backward
        {"name": "norm_rope_train", "op": "norm_rope", "tokens": 8191, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": "halves",
         "norm": True, "train": True, "type": "bf16"},
        # one decoded token's keys and values into the cache
        {"name": "append_1", "op": "append", "tokens": 1, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": "interleaved", "norm": False, "page": 64,
         "skip": 0.0, "type": "f32"},
        # a padded batch of decoded tokens, each of a sequence of its own
        {"name": "append_33", "op": "append", "tokens": 33, "kv_heads": 12, "dim": 64, "rot": 64, "pairs": "halves", "norm": True, "page": 16,
         "skip": 0.2, "type": "f16"},
        # a long prompt
        {"name": "append_8192", "op": "append", "tokens": 8192, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": "halves", "norm": True, "page": 64,
         "skip": 0.01, "type": "bf16"},
        # one sequence decoding after a short prompt
        {"name": "attend_1", "op": "attend", "seqs": 1, "queries": 1, "cached": 1023, "ragged": False, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "window": 0, "type": "f32"},
        # a few sequences with some drafted tokens each, a head of its own for every query head
        {"name": "attend_7x3", "op": "attend", "seqs": 7, "queries": 3, "cached": 1021, "ragged": True, "q_heads": 12, "kv_heads": 12, "dim": 64,
         "page": 16, "window": 0, "type": "f32"},
        # a serving batch of ragged contexts
        {"name": "attend_64", "op": "attend", "seqs": 64, "queries": 1, "cached": 8192, "ragged": True, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "window": 0, "type": "bf16"},
        # one very long context
        {"name": "attend_long", "op": "attend", "seqs": 1, "queries": 1, "cached": 131072, "ragged": False, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 256, "window": 0, "type": "f16"},
        # a chunk of a long prompt behind what is cached already
        {"name": "attend_chunk", "op": "attend", "seqs": 1, "queries": 512, "cached": 8192, "ragged": False, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "window": 0, "type": "bf16"},
        # two prompts of their own, with a sliding window
        {"name": "attend_prompts", "op": "attend", "seqs": 2, "queries": 2048, "cached": 2048, "ragged": True, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 32, "window": 1024, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    heads = rng.choice([(32, 8), (12, 12), (16, 4), (24, 3), (8, 1), (10, 2), (28, 4)])
    c = {"op": op, "type": rng.choice(["f32", "f16", "bf16"]), "kv_heads": heads[1], "dim": rng.choice([64, 96, 128, 128])}
    if op != "attend":
        c |= {"tokens": _log(rng, 1, 8192), "pairs": rng.choice(["halves", "interleaved"]), "norm": rng.random() < 0.6}
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2])
    if op == "norm_rope":
        c |= {"q_heads": heads[0], "train": rng.random() < 0.5}
    elif op == "append":
        c |= {"page": rng.choice([16, 32, 64, 256]), "skip": rng.choice([0.0, 0.1])}
    else:
        c |= {"q_heads": heads[0], "page": rng.choice([16, 32, 64, 256]), "ragged": rng.random() < 0.6, "queries": _log(rng, 1, 1024)}
        if rng.random() < 0.4:
            c["queries"] = 1
        c["cached"] = max(c["queries"], _log(rng, 16, 65536))
        c["seqs"] = _log(rng, 1, 100)
        while c["seqs"] > 1 and (c["seqs"] * c["cached"] > 1 << 18 or c["seqs"] * c["cached"] * c["queries"] > 1 << 22):
            c["seqs"] //= 2
        while c["cached"] * c["queries"] > 1 << 22:
            c["queries"] = c["queries"] // 2 + 1
        c["window"] = rng.choice([0, 0, 257])
    return c


def _lengths(case):
    """(queries, cached tokens) of each sequence: all alike, or spread evenly down to a small share."""
    n = case["seqs"]
    if not case["ragged"]:
        return [(case["queries"], case["cached"])] * n
    got = []
    for i in range(n):
        share = 1.0 - i * 0.9 / max(1, n)
        q = max(1, round(case["queries"] * share))
        got.append((q, max(q, round(case["cached"] * (1.0 - ((i * 7) % n) * 0.9 / n)))))
    return got


def work(case):
    t, d, kv = BYTES[case["type"]], case["dim"], case["kv_heads"]
    if case["op"] == "attend":
        pairs = keys = rows = 0
        for q, cached in _lengths(case):
            seen = [min(case["window"] or cached, cached - q + i + 1) for i in range(q)]
            pairs += sum(seen)
            keys += min(cached, (case["window"] or cached) + q - 1)
            rows += q
        return {"bytes": keys * kv * d * 2 * 9 / 16 + 2 * rows * case["q_heads"] * d * t, "flops": 4 * d * case["q_heads"] * pairs}
    n = case["tokens"]
    table = n * (8 + 4 * case["rot"])
    if case["op"] == "norm_rope":
        values = n * (case["q_heads"] + kv) * d
        return {"bytes": values * t * (5 if case["train"] else 2) + table, "flops": values * (25 if case["train"] else 8)}
    values = 2 * n * kv * d
    return {"bytes": values * (2 * t + 9 / 8) + table, "flops": values * 12}      # in; codes out and in again; values out


# ------------------------------------------------------------------ inputs --

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _heads(g, n, heads, dim):
    """Rows of heads with one channel in thirty larger, as keys and queries have them."""
    x = _normal(g, n, heads, dim)
    return x * torch.where(torch.rand(heads, dim, generator=g, device=DEV) < 0.03, 6.0, 1.0)


def _table(n_pos, rot, base=500000.0):
    """Cosines and sines of the positions' angles, fp32 [positions, rot]: rot / 2 of each."""
    angle = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s, t, d, kv = dict(case), TYPES[case["type"]], case["dim"], case["kv_heads"]
    if case["op"] == "attend":
        lengths = _lengths(case)
        need = [-(-c // case["page"]) for _, c in lengths]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).int()
        table, at = torch.full((len(need), max(need)), -1, dtype=torch.int32, device=DEV), 0
        slots = []
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
            j = torch.arange(lengths[i][1], device=DEV)
            slots.append(table[i].long()[j // case["page"]] * case["page"] + j % case["page"])
        slots = torch.cat(slots)
        s["cache"] = torch.randint(0, 256, (pages, kv * case["page"] * d * 9 // 8), generator=g, device=DEV, dtype=torch.uint8)
        _put(s["cache"], case["page"], slots, _heads(g, slots.numel(), kv, d), _heads(g, slots.numel(), kv, d))
        rows = sum(q for q, _ in lengths)
        qkv = torch.empty(rows, (case["q_heads"] + 2 * kv) * d, dtype=t, device=DEV)
        qkv[:, : case["q_heads"] * d] = _heads(g, rows, case["q_heads"], d).reshape(rows, -1)
        s["q"] = qkv[:, : case["q_heads"] * d].unflatten(1, (case["q_heads"], d))
        s["pages"] = table
        s["len"] = torch.tensor([c for _, c in lengths], dtype=torch.int32, device=DEV)
        s["first"] = torch.tensor([0] + [q for q, _ in lengths], device=DEV).cumsum(0).int()
        s["most"] = max(q for q, _ in lengths)
        return s
    n, positions = case["tokens"], 32768
    q_heads = case.get("q_heads", 0)
    qkv = torch.cat((_heads(g, n, q_heads + kv, d).reshape(n, -1), _normal(g, n, kv * d)), 1).to(t)
    s["q"] = qkv[:, : q_heads * d].unflatten(1, (q_heads, d)) if q_heads else None
    s["k"] = qkv[:, q_heads * d: (q_heads + kv) * d].unflatten(1, (kv, d))
    s["v"] = qkv[:, (q_heads + kv) * d:].unflatten(1, (kv, d))
    s["table"] = _table(positions, case["rot"])
    start = int(torch.randint(0, positions - n, (), generator=g, device=DEV))
    s["pos"] = (torch.arange(n, device=DEV) + start).int() if n > 100 else torch.randint(0, positions, (n,), generator=g, device=DEV).int()
    s["qw"] = 1 + 0.2 * _normal(g, d) if case["norm"] else None
    s["kw"] = 1 + 0.2 * _normal(g, d) if case["norm"] else None
    if case["op"] == "norm_rope":
        if case["train"]:
            s["gq"], s["gk"] = _normal(g, n, q_heads, d).to(t), _normal(g, n, kv, d).to(t)
        return s
    page = case["page"]
    pages = -(-n // page) + 2                                                                            # the last one is nobody's
    s["cache"] = torch.randint(0, 256, (pages, kv * page * d * 9 // 8), generator=g, device=DEV, dtype=torch.uint8)
    order = torch.randperm(pages - 1, generator=g, device=DEV)
    j = torch.arange(n, device=DEV) + page // 2
    slots = order[j // page] * page + j % page
    s["slots"] = torch.where(torch.rand(n, generator=g, device=DEV) < case["skip"], -1, slots).int()
    return s


# ------------------------------------------------------------- plain forms --

def _rotated(z, table, pos, pairs):
    """fp32 [tokens, heads, D] with its first values rotated by the angles of their positions."""
    half = table.shape[1] // 2
    c, s = table[pos.long()][:, None].split(half, -1)
    if pairs == "halves":
        a, b = z[..., :half], z[..., half: 2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = z[..., 0: 2 * half: 2], z[..., 1: 2 * half: 2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((turned, z[..., 2 * half:]), -1)


def _inverse_norm(x):
    return (1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + EPS)).float()


def _norm_rope(x, w, s):
    z = x.float()
    return _rotated(z if w is None else z * _inverse_norm(z) * w, s["table"], s["pos"], s["pairs"])


def _norm_rope_back(g, x, w, s):
    """The gradients of _norm_rope for its row and its weight."""
    t = torch.cat((s["table"][:, : s["rot"] // 2], -s["table"][:, s["rot"] // 2:]), 1)
    dz = _rotated(g.float(), t, s["pos"], s["pairs"])
    if w is None:
        return dz, None
    r = _inverse_norm(x.float())
    xh, dh = x.float() * r, dz * w
    return r * (dh - xh * (dh * xh).mean(-1, keepdim=True)), (dz * xh).double().sum((0, 1)).float()


def _codes(x):
    """fp32 [..., D] -> codes 0 to 15 [..., D / 32, 32] and scales fp16 [..., D / 32]."""
    b = x.clamp(-65504, 65504).unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 8
    v = (b / torch.where(d > 0, d, torch.ones_like(d))).double()
    code = (torch.sign(v) * torch.floor(v.abs() + 0.5)).clamp(-8, 7)
    return (code + 8).to(torch.uint8), d[..., 0].half()


def _bytes_of(nibbles):
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)


def _chunks(cache, page):
    """The chunks of a cache [pages, bytes] with their tokens: [pages, kv heads, page / 16, 18 D], D from the caller."""
    return lambda d: cache.view(cache.shape[0], -1, page // 16, 18 * d)


def _put(cache, page, slots, k, v):
    """Encode keys and values fp32 [tokens, kv heads, D] into their slots."""
    n, heads, d = k.shape
    blocks, flat = d // 32, _chunks(cache, page)(d)
    p, group, token = slots // page, slots % page // 16, slots % 16
    head = torch.arange(heads, device=cache.device)
    kc, ks = _codes(k)
    vc, vs = _codes(v)
    kb = _bytes_of(kc.unflatten(-1, (4, 8)).transpose(-3, -2).contiguous()).flatten(-3)                  # [t][b] words
    vb = _bytes_of(vc.unflatten(-1, (8, 4)).transpose(-3, -2).contiguous())                              # [g][b] halves
    index = (p[:, None], head[None], group[:, None])
    i = torch.arange(d // 2, device=cache.device)
    put = lambda start, where, value: flat.index_put_((*(x[..., None] for x in index), start + where), value)  # noqa: E731
    put(0, token[:, None, None] * (d // 2) + i, kb)
    g, b, byte = i // (2 * blocks), i // 2 % blocks, i % 2
    octet, pair, odd = (x[:, None, None] for x in (token // 8, token // 2 % 4, token % 2))
    put(8 * d, octet * 4 * d + ((g * 4 + pair) * blocks + b) * 4 + odd * 2 + byte, vb.flatten(-3))
    j = torch.arange(2 * blocks, device=cache.device)
    put(16 * d, token[:, None, None] * (2 * blocks) + j, ks.contiguous().view(torch.uint8))
    put(17 * d, token[:, None, None] * (2 * blocks) + j, vs.contiguous().view(torch.uint8))


def _decoded(chunk, d):
    """Chunks [..., 18 D] -> keys and values fp32 [..., 16, D]."""
    blocks, lead = d // 32, chunk.shape[:-1]
    nibbles = lambda c: torch.stack((c & 15, c >> 4), -1).flatten(-2).float() - 8  # noqa: E731
    kc = nibbles(chunk[..., : 8 * d].reshape(*lead, 16, 4, blocks, 4)).transpose(-3, -2).flatten(-2)
    vc = nibbles(chunk[..., 8 * d: 16 * d].reshape(*lead, 2, 8, 4, blocks, 2, 2))                        # o g p b e n
    n = len(lead)
    vc = vc.permute(*range(n), n, n + 2, n + 4, n + 3, n + 1, n + 5).reshape(*lead, 16, blocks, 32)
    scales = chunk[..., 16 * d:].contiguous().view(torch.float16).reshape(*lead, 2, 16, blocks, 1).float()
    return (kc * scales[..., 0, :, :, :]).flatten(-2), (vc * scales[..., 1, :, :, :]).flatten(-2)


def _plain_norm_rope(s):
    t = TYPES[s["type"]]
    out = {"q": _norm_rope(s["q"], s["qw"], s).to(t), "k": _norm_rope(s["k"], s["kw"], s).to(t)}
    if s["train"]:
        dq, dqw = _norm_rope_back(s["gq"], s["q"], s["qw"], s)
        dk, dkw = _norm_rope_back(s["gk"], s["k"], s["kw"], s)
        out |= {"dq": dq.to(t), "dk": dk.to(t), "dqw": dqw, "dkw": dkw}
    return out


def _plain_append(s):
    t, d, kept = TYPES[s["type"]], s["dim"], s["slots"] >= 0
    at = torch.where(kept, s["slots"], s["cache"].shape[0] * s["page"] - 1).long()                        # what is skipped goes to the spare page
    kept = kept[:, None, None]
    _put(s["cache"], s["page"], at, _norm_rope(s["k"], s["kw"], s), s["v"].float())
    k, v = _read(s["cache"], s["page"], at, d)
    return {"k": torch.where(kept, k, 0.0).to(t), "v": torch.where(kept, v, 0.0).to(t)}


def _read(cache, page, slots, d):
    chunk = _chunks(cache, page)(d)[slots // page, :, slots % page // 16]
    k, v = _decoded(chunk, d)
    at = (torch.arange(slots.numel(), device=slots.device), slice(None), slots % 16)
    return k[at], v[at]


def _plain_attend(s):
    n, d, kv = s["len"].numel(), s["dim"], s["kv_heads"]
    k, v = _decoded(_chunks(s["cache"], s["page"])(d)[s["pages"].long().clamp(min=0)], d)                # [n, pages, kv, groups, 16, D]
    k, v = (x.transpose(1, 2).flatten(2, 4) for x in (k, v))                                             # [n, kv, keys, D]
    j = torch.arange(k.shape[2], device=DEV)
    here = j < s["len"][:, None]
    k, v = (torch.where(here[:, None, :, None], x, 0.0) for x in (k, v))
    first, count = s["first"][:-1].long(), s["first"][1:] - s["first"][:-1]
    i = torch.arange(s["most"], device=DEV)
    row = torch.where(i < count[:, None], first[:, None] + i, 0)
    q = s["q"].float()[row].unflatten(2, (kv, -1)).permute(0, 2, 3, 1, 4)                                 # [n, kv, shared, queries, D]
    scores = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, q.shape[2:4]) * d ** -0.5
    last = (s["len"] - count)[:, None] + i                                                               # the last key that query i sees
    seen = (j <= last[..., None]) & here[:, None]
    if s["window"]:
        seen &= j > last[..., None] - s["window"]
    scores = torch.where(seen[:, None, None], scores, -torch.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -torch.inf, top, 0.0))
    o = (p.flatten(2, 3) @ v).unflatten(2, q.shape[2:4]) / p.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[i < count[:, None]].to(TYPES[s["type"]])


# ---------------------------------------------------------- the operators ---

def _own_norm_rope(s):
    import q4_quantized_matmul_gb300 as q4q
    mode = q4q.Q4Q_ROPE_HALVES if s["pairs"] == "halves" else q4q.Q4Q_ROPE_PAIRS
    args = {"q_weight": s["qw"], "k_weight": s["kw"], "eps": EPS, "table": s["table"], "pos": s["pos"], "mode": mode}
    out = dict(zip("qk", q4q.q4q_qk_norm_rope(s["q"], s["k"], **args)))
    if s["train"]:
        out |= dict(zip(("dq", "dk", "dqw", "dkw"), q4q.q4q_qk_norm_rope_back(s["gq"], s["gk"], s["q"], s["k"], **args)))
    return out


def _own_append(s):
    import q4_quantized_matmul_gb300 as q4q
    mode = q4q.Q4Q_ROPE_HALVES if s["pairs"] == "halves" else q4q.Q4Q_ROPE_PAIRS
    q4q.q4q_kv_append(s["cache"], s["page"], s["k"], s["v"], s["slots"], k_weight=s["kw"], eps=EPS, table=s["table"], pos=s["pos"], mode=mode)
    k, v = q4q.q4q_kv_get_rows(s["cache"], s["page"], s["kv_heads"], s["dim"], s["slots"], dst_dtype=TYPES[s["type"]])
    return {"k": k, "v": v}


def _own_attend(s):
    import q4_quantized_matmul_gb300 as q4q
    return q4q.q4q_kv_attn(s["q"], s["cache"], s["page"], s["kv_heads"], s["pages"], s["len"], first=s["first"], window=s["window"])


def run(state):
    op = state["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "append": _own_append, "attend": _own_attend}[op](state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "attend": _plain_attend}[op](state)


# ------------------------------------------------------ 64-bit definitions --

def _single(x):
    """64-bit values rounded to fp32 where the definition rounds."""
    return x.float().double()


def _turned64(z, table, pos, interleaved, rounding):
    out, half = z.clone(), table.shape[1] // 2
    i = torch.arange(half, device=z.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    rows = table.double().index_select(0, pos.long()).unsqueeze(1)
    c, s = rows[..., :half], rows[..., half:]
    out[..., a] = rounding(rounding(z[..., a] * c) - rounding(z[..., b] * s))
    out[..., b] = rounding(rounding(z[..., b] * c) + rounding(z[..., a] * s))
    return out


def _normed64(x, w):
    x = x.double()
    if w is None:
        return x
    r = _single((torch.einsum("thd,thd->th", x, x) / x.shape[-1] + EPS) ** -0.5)[..., None]
    return _single(_single(x * r) * w.double())


def _block_values64(x):
    """The values that Q4_0 blocks of x hold."""
    lim = x.clamp(-65504.0, 65504.0).reshape(*x.shape[:-1], -1, 32)
    d = lim.abs().max(-1, keepdim=True).values / 8
    q = torch.nan_to_num(_single(lim / d))
    q = torch.where(q < 0, torch.ceil(q - 0.5), torch.floor(q + 0.5)).clamp(-8, 7)
    return (q * d.half().double()).reshape(x.shape)


def _cached64(cache, page, heads, d, slots):
    """Keys and values [slots, heads, D] in 64 bits, each value looked up by its own address."""
    flat, blocks = cache.view(-1), d // 32
    token, dim = slots % 16, torch.arange(d, device=cache.device)
    chunk = ((slots // page)[:, None] * heads + torch.arange(heads, device=cache.device)) * (page // 16) + (slots % page // 16)[:, None]
    b, in_block, token = dim // 32, dim % 32, token[:, None]
    places = (token * (d // 2) + (in_block // 8 * blocks + b) * 4 + in_block % 8 // 2,
              8 * d + token // 8 * 4 * d + ((in_block // 4 * 4 + token // 2 % 4) * blocks + b) * 4 + token % 2 * 2 + in_block % 4 // 2)
    got = []
    for i, place in enumerate(places):
        byte = flat[(chunk * 18 * d)[..., None] + place[:, None]].int()
        code = torch.where(dim % 2 == 1, byte >> 4, byte & 15) - 8
        scale = cache.view(torch.float16).view(-1)[(chunk * 9 * d)[..., None] + (16 + i) * d // 2 + (token * blocks + b)[:, None]]
        got.append(code.double() * scale.double())
    return got


def _gradients64(g, x, w, s):
    x, g = x.double(), g.double()
    back = torch.cat((s["table"][:, : s["rot"] // 2], -s["table"][:, s["rot"] // 2:]), 1)
    dz = _turned64(g, back, s["pos"], s["pairs"] == "interleaved", lambda v: v)
    if w is None:
        return dz, None
    m = torch.einsum("thd,thd->th", x, x)[..., None] / x.shape[-1] + EPS
    dh = dz * w.double()
    dx = dh * m ** -0.5 - x * (dh * x).sum(-1, keepdim=True) / x.shape[-1] * m ** -1.5
    return dx, torch.einsum("thd,thd->d", dz, x * m ** -0.5)


def exact(case, seed):
    s = prepare(case, seed)
    interleaved = case.get("pairs") == "interleaved"
    if case["op"] == "norm_rope":
        out = {n: _turned64(_normed64(s[n], s[n + "w"]), s["table"], s["pos"], interleaved, _single) for n in "qk"}
        if case["train"]:
            for n in "qk":
                out["d" + n], out["d%sw" % n] = _gradients64(s["g" + n], s[n], s[n + "w"], s)
        return out
    if case["op"] == "append":
        kept = (s["slots"] >= 0).double()[:, None, None]
        k = _turned64(_normed64(s["k"], s["kw"]), s["table"], s["pos"], interleaved, _single)
        return {"k": _block_values64(k) * kept, "v": _block_values64(s["v"].double()) * kept}
    d, kv, outs = case["dim"], case["kv_heads"], []
    shared = case["q_heads"] // kv
    for i, (n, cached) in enumerate(_lengths(case)):
        j = torch.arange(cached, device=DEV)
        slots = s["pages"][i].long()[j // case["page"]] * case["page"] + j % case["page"]
        k, v = _cached64(s["cache"], case["page"], kv, d, slots)
        q = s["q"][s["first"][i]: s["first"][i + 1]].double()
        last = torch.arange(n, device=DEV)[:, None] + cached - n
        hidden = (j > last) | ((j <= last - case["window"]) if case["window"] else torch.zeros_like(j > last))
        o = torch.empty_like(q)
        for h in range(case["q_heads"]):
            scores = (q[:, h] @ k[:, h // shared].T / d ** 0.5).masked_fill(hidden, -torch.inf)
            o[:, h] = torch.softmax(scores, -1) @ v[:, h // shared]
        outs.append(o)
    return torch.cat(outs)
