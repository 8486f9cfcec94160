"""Cases of the MXFP4 operators: block encoding, the weight product, tokens sorted by expert and the experts' products.

MXFP4 holds 32 values in 16 bytes of E2M1 codes and one E8M0 scale.  For a block with largest magnitude amax
    e = floor(log2(amax)) - 2,   value = 2^e * E2M1(x * 2^-e)   (nearest, ties to the even code, at most 6),
and e = -127 for a block of zeros.  Activations are encoded on the fly, to MXFP4 in the same way or to MXFP8 with
    e = floor(log2(amax)) - 8,   value = 2^e * E4M3(x * 2^-e)   (nearest, ties to even, at most 448).
One matrix [rows, K] is one buffer: the code plane, rows of Kp / 2 bytes (Kp: K rounded up to 256, low nibble first),
rounded up to 256 bytes; then the scale plane, for each 128 rows x 128 columns 512 bytes with the scale of row r and
block b at (r % 32) * 16 + (r / 32 % 4) * 4 + b % 4.  Codes of the columns past K, and scales past the matrix, are 0.
"""
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a feed-forward matrix encoded when a checkpoint is loaded, and read back
        {"name": "encode_ffn", "op": "encode", "k": 4096, "rows": 14336, "type": "f32", "lookups": 512},
        # a token-embedding table with an odd number of rows, and the lookups of a prompt
        {"name": "encode_vocab", "op": "encode", "k": 768, "rows": 50257, "type": "bf16", "lookups": 77},
        # one token of a decode step through the up projection
        {"name": "product_1", "op": "product", "k": 4096, "rows": 14336, "tokens": 1, "acts": "mxfp8", "type": "f32"},
        # a few sequences decoded together through an lm_head with an odd vocabulary
        {"name": "product_7_lm_head", "op": "product", "k": 768, "rows": 50257, "tokens": 7, "acts": "mxfp4", "type": "f16"},
        # an odd batch through the down projection, where few row tiles meet a long K
        {"name": "product_33", "op": "product", "k": 14336, "rows": 4096, "tokens": 33, "acts": "mxfp8", "type": "bf16"},
        # a prompt through the up projection
        {"name": "product_512", "op": "product", "k": 4096, "rows": 14336, "tokens": 512, "acts": "mxfp8", "type": "bf16"},
        # a long prompt in 4-bit activations
        {"name": "product_2048", "op": "product", "k": 14336, "rows": 4096, "tokens": 2048, "acts": "mxfp4", "type": "f32"},
        # one decoded token routed and its experts' answers weighted
        {"name": "route_1", "op": "route", "k": 4096, "tokens": 1, "top": 2, "experts": 8, "type": "f32", "train": False, "drop": False},
        # a training batch sorted by expert and back, forward and backward, some choices dropped
        {"name": "route_train", "op": "route", "k": 2048, "tokens": 8191, "top": 4, "experts": 64, "type": "bf16", "train": True, "drop": True},
        # three decoded tokens through the up projections of their experts
        {"name": "experts_3", "op": "experts", "k": 4096, "rows": 14336, "tokens": 3, "top": 2, "experts": 8, "acts": "mxfp8", "type": "f32", "drop": False},
        # many small experts with ragged sizes
        {"name": "experts_ragged", "op": "experts", "k": 1504, "rows": 777, "tokens": 517, "top": 4, "experts": 32, "acts": "mxfp8", "type": "bf16", "drop": True},
        # a prompt through the up projections of its experts
        {"name": "experts_2048", "op": "experts", "k": 4096, "rows": 14336, "tokens": 2048, "top": 2, "experts": 8, "acts": "mxfp4", "type": "bf16", "drop": False},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _size(rng, lo, hi, step=1):
    v = max(lo, _log(rng, lo, hi) // step * step)
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["encode", "product", "product", "route", "experts", "experts"])
    c = {"op": op, "type": rng.choice(["f32", "f16", "bf16"])}
    if op == "encode":
        c |= {"k": _size(rng, 256, 14336, 32), "rows": _size(rng, 64, 50257), "lookups": _size(rng, 1, 512)}
    elif op == "product":
        c |= {"k": _size(rng, 256, 14336, 32), "rows": _size(rng, 64, 50257), "tokens": _size(rng, 1, 2048), "acts": rng.choice(["mxfp4", "mxfp8"])}
    elif op == "route":
        c |= {"k": _size(rng, 64, 4096, 8), "tokens": _size(rng, 1, 8192), "experts": _size(rng, 4, 256), "train": rng.random() < 0.5, "drop": rng.random() < 0.5}
        c["top"] = rng.choice([1, 2, 4])
    else:
        c |= {"k": _size(rng, 256, 4096, 32), "rows": _size(rng, 64, 14336), "tokens": _size(rng, 1, 2048), "experts": _size(rng, 4, 64)}
        c |= {"top": rng.choice([1, 2, 4]), "acts": rng.choice(["mxfp4", "mxfp8"]), "drop": rng.random() < 0.5}
    while c.get("rows", 0) * c["k"] * c.get("experts", 1) > 1 << (28 if op == "experts" else 26):
        c["rows"] = c["rows"] // 2 + 1
    if c.get("rows") == 3072:
        c["rows"] += 1
    return c


def work(case):
    k, t, op = case["k"], BYTES[case["type"]], case["op"]
    if op == "encode":
        packed = case["rows"] * k * 17 / 32
        return {"bytes": case["rows"] * k * (t + 4) + packed + case["lookups"] * (4 + k * (17 / 32 + 4)), "flops": 0}
    if op == "product":
        n, m = case["tokens"], case["rows"]
        return {"bytes": m * k * 17 / 32 + n * (k + m) * t, "flops": 2 * m * n * k}
    n, slots = case["tokens"], case["tokens"] * case["top"]
    if op == "route":
        moved = 3 * 4 * slots + 4 * slots + t * k * (2 * n + 2 * slots)    # ids, places, weights; x, y; sorted rows, experts' rows
        if case["train"]:
            moved += t * k * (2 * n + 2 * slots) + 4 * slots               # dy, dx; the sorted rows' gradient in and out; dw
        return {"bytes": moved, "flops": 2 * slots * k * (3 if case["train"] else 1)}
    m, busy = case["rows"], min(case["experts"], slots)
    return {"bytes": busy * m * k * 17 / 32 + t * (n * k + slots * m) + 4 * slots, "flops": 2 * slots * m * k}


# ------------------------------------------------------------------ inputs --

def _up(v, m):
    return (v + m - 1) // m * m


def _floor_log2(a):
    """floor(log2(a)) of positive normal fp32 values, from their bits."""
    return (a.contiguous().view(torch.int32) >> 23) - 127


def _two_to(e):
    """2^e as fp32, -127 <= e <= 127."""
    return torch.where(e == -127, torch.full((), 2.0 ** -127, device=e.device), ((e.clamp(min=-126) + 127) << 23).view(torch.float32))


def _blocks(x, top):
    """fp32 [rows, K] -> its blocks [rows, K / 32, 32] and their exponents, `top` the element type's largest exponent."""
    b = x.float().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    return b, torch.where(amax > 0, _floor_log2(amax) - top, torch.full_like(amax, -127, dtype=torch.int32)).clamp(min=-127)


def _e2m1(v):
    a = v.abs()
    step = _two_to(_floor_log2(a.clamp(min=1.0)) - 1)
    return torch.where(v < 0, -1.0, 1.0) * (torch.round(a / step) * step).clamp(max=6.0)


def _e4m3(v):
    a = v.abs()
    step = _two_to(_floor_log2(a.clamp(min=2.0 ** -6)) - 3)
    return torch.where(v < 0, -1.0, 1.0) * (torch.round(a / step) * step).clamp(max=448.0)


def _encoded(x, acts):
    """The values that the encoding of the rows of `x` stands for, fp32."""
    b, e = _blocks(x, 2 if acts == "mxfp4" else 8)
    e = e[..., None]
    v = b * _two_to(-e)
    return ((_e2m1(v) if acts == "mxfp4" else _e4m3(v)) * _two_to(e)).reshape(x.shape)


def _pack(w):
    """fp32 [rows, K] -> the buffer of one MXFP4 matrix (see the module's text)."""
    rows, k = w.shape
    kp = _up(k, 256)
    b, e = _blocks(w, 2)
    v = _e2m1(b * _two_to(-e[..., None])).reshape(rows, k)
    a = v.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    nib = torch.zeros((rows, kp), dtype=torch.uint8, device=w.device)
    nib[:, :k] = code
    codes = (nib[:, 0::2] | (nib[:, 1::2] << 4)).reshape(-1)
    sc = torch.zeros((_up(rows, 128), kp // 32), dtype=torch.uint8, device=w.device)
    sc[:rows, : k // 32] = (e + 127).to(torch.uint8)
    scales = sc.reshape(-1, 4, 32, kp // 128, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    out = torch.zeros(_up(codes.numel(), 256) + scales.numel(), dtype=torch.uint8, device=w.device)
    out[: codes.numel()] = codes
    out[-scales.numel():] = scales
    return out


def _unpacked(buf, rows, k):
    """E2M1 values [rows, K] fp32 and scale bytes [rows, K / 32] of one packed matrix, or of several ([..., bytes])."""
    kp, lead = _up(k, 256), buf.shape[:-1]
    codes = buf[..., : rows * kp // 2].reshape(*lead, rows, kp // 2)
    n_sc = _up(rows, 128) * kp // 32
    grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=buf.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).reshape(*lead, rows, kp)[..., :k].int()]
    d = len(lead)
    sc = buf[..., buf.shape[-1] - n_sc:].reshape(*lead, -1, kp // 128, 32, 4, 4).permute(*range(d), d, d + 3, d + 2, d + 1, d + 4)
    return v, sc.reshape(*lead, -1, kp // 32)[..., :rows, : k // 32].int()


def _decoded(buf, rows, k):
    v, s = _unpacked(buf, rows, k)
    return v * _two_to(s - 127).repeat_interleave(32, -1)


def _normal(g, *shape, scale=1.0, type="f32"):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(TYPES[type])


def _weights(g, rows, k):
    """Normal weights with a few large ones and some blocks of zeros."""
    w = _normal(g, rows, k, scale=0.02)
    w *= torch.where(torch.rand(rows, k, generator=g, device=DEV) < 0.001, 20.0, 1.0)
    return (w.reshape(rows, -1, 32) * (torch.rand(rows, k // 32, 1, generator=g, device=DEV) > 0.01)).reshape(rows, k)


def _acts(g, n, k, type):
    """Normal activations with one channel in a hundred ten times as large."""
    return (_normal(g, n, k) * torch.where(torch.rand(k, generator=g, device=DEV) < 0.01, 10.0, 1.0)).to(TYPES[type])


def _ids(g, n, top, experts, drop):
    """A router's choices: distinct experts for each token, some more popular than others; dropped choices are -1."""
    logits = _normal(g, n, experts) + 0.7 * _normal(g, 1, experts)
    top = min(top, experts)
    ids = logits.topk(top, dim=1).indices.to(torch.int32)
    if drop:
        ids = torch.where(torch.rand(n, top, generator=g, device=DEV) < 0.05, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s, k, op, t = dict(case), case["k"], case["op"], case["type"]
    if op == "encode":
        s["w"] = _weights(g, case["rows"], k).to(TYPES[t])
        s["ids"] = torch.randint(0, case["rows"], (case["lookups"],), generator=g, device=DEV, dtype=torch.int32)
        return s
    n = case["tokens"]
    s["x"] = _acts(g, n, k, t)
    if op == "product":
        s["w"] = _pack(_weights(g, case["rows"], k))
        return s
    s["ids"] = _ids(g, n, case["top"], case["experts"], case["drop"])
    if op == "experts":
        s["w"] = torch.stack([_pack(_weights(g, case["rows"], k)) for _ in range(case["experts"])])
        return s
    slots = s["ids"].numel()
    s["rows"] = _normal(g, slots, k, type=t)
    s["weights"] = torch.softmax(_normal(g, *s["ids"].shape), -1)
    if case["train"]:
        s["dy"] = _normal(g, n, k, type=t)
        s["dsorted"] = _normal(g, slots, k, type=t)
    return s


# ------------------------------------------------------------- plain forms --

def _sorted(ids, experts):
    """Choices in the order of their expert, dropped ones last: (first row of each expert, slot of each row, row of each slot)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    slot = torch.argsort(key, stable=True)
    row = torch.empty_like(slot)
    row[slot] = torch.arange(slot.numel(), device=slot.device)
    count = (key[None, :] == torch.arange(experts, device=key.device)[:, None]).sum(1)
    first = torch.cat((torch.zeros(1, dtype=torch.long, device=key.device), torch.cumsum(count, 0)))
    return first, slot, row


def _plain_encode(s):
    w = _encoded(s["w"], "mxfp4")
    return {"values": w, "looked_up": w[s["ids"].long()]}


def _plain_product(s):
    y = _encoded(s["x"], s["acts"]) @ _decoded(s["w"], s["rows"], s["k"]).T
    return y.to(TYPES[s["type"]])


def _plain_experts(s):
    first, slot, _ = _sorted(s["ids"], s["experts"])
    count = first[1:] - first[:-1]
    place = torch.arange(int(count.max()) if count.numel() else 0, device=first.device)
    at = (first[:-1, None] + place).clamp(max=slot.numel() - 1)              # [experts, most rows of one expert]
    here = place < count[:, None]
    x = _encoded(s["x"], s["acts"])[slot[at] // s["ids"].shape[1]]
    y = torch.bmm(x, _decoded(s["w"], s["rows"], s["k"]).transpose(1, 2))
    out = torch.zeros((slot.numel(), s["rows"]), device=y.device)
    out[at[here]] = y[here]
    return {"first": first.int(), "row": _sorted(s["ids"], s["experts"])[2].int(), "out": out.to(TYPES[s["type"]])}


def _plain_route(s):
    first, slot, row = _sorted(s["ids"], s["experts"])
    n, top = s["ids"].shape
    t, kept = TYPES[s["type"]], first[-1]
    token = slot // top
    here = (torch.arange(slot.numel(), device=slot.device) < kept)[:, None]
    place = row.reshape(n, top)
    used = (place < kept)[..., None]
    w = torch.where(used, s["weights"][..., None], 0.0)
    answers = torch.where(used, s["rows"].float()[place], 0.0)
    out = {"first": first.int(), "row": row.int(), "sorted": torch.where(here, s["x"][token], 0.0).to(t), "y": (w * answers).sum(1).to(t)}
    if s["train"]:
        dy = s["dy"].float()
        out["drows"] = torch.where(here, (s["weights"].reshape(-1)[slot])[:, None] * dy[token], 0.0).to(t)
        out["dweights"] = (answers * dy[:, None]).sum(-1)
        out["dx"] = torch.where(used, s["dsorted"].float()[place], 0.0).sum(1).to(t)
    return out


# ---------------------------------------------------------- the operators ---

def _own_encode(s):
    import q4_quantized_matmul_gb300 as q4q
    w = q4q.q4q_quantize_mxfp4(s["w"])
    return {"values": q4q.q4q_get_rows_mxfp4(w, s["k"], s["rows"]),
            "looked_up": q4q.q4q_get_rows_mxfp4(w, s["k"], s["rows"], s["ids"])}


def _own_product(s):
    import q4_quantized_matmul_gb300 as q4q
    acts = q4q.Q4Q_ACTS_MXFP4 if s["acts"] == "mxfp4" else q4q.Q4Q_ACTS_MXFP8
    return q4q.q4q_mul_mat_mxfp4(s["w"], s["k"], s["rows"], s["x"], acts)


def _own_experts(s):
    import q4_quantized_matmul_gb300 as q4q
    acts = q4q.Q4Q_ACTS_MXFP4 if s["acts"] == "mxfp4" else q4q.Q4Q_ACTS_MXFP8
    first, slot, row = q4q.q4q_moe_sort(s["ids"], s["experts"])
    return {"first": first, "row": row, "out": q4q.q4q_mul_mat_id_mxfp4(s["w"], s["k"], s["rows"], s["x"], first, slot, s["ids"].shape[1], acts)}


def _own_route(s):
    import q4_quantized_matmul_gb300 as q4q
    first, slot, row = q4q.q4q_moe_sort(s["ids"], s["experts"])
    out = {"first": first, "row": row, "sorted": q4q.q4q_moe_gather(s["x"], first, row, s["ids"].shape[1]),
           "y": q4q.q4q_moe_combine(s["rows"], first, row, s["weights"])}
    if s["train"]:
        out["drows"], out["dweights"] = q4q.q4q_moe_combine_back(s["dy"], s["rows"], first, row, s["weights"])
        out["dx"] = q4q.q4q_moe_gather_back(s["dsorted"], first, row, s["ids"].shape[1])
    return out


def run(state):
    op = state["op"]
    if own:
        return {"encode": _own_encode, "product": _own_product, "experts": _own_experts, "route": _own_route}[op](state)
    return {"encode": _plain_encode, "product": _plain_product, "experts": _plain_experts, "route": _plain_route}[op](state)


# ------------------------------------------------------ 64-bit definitions --

def _nearest(a, grid):
    """The nearest of `grid`'s values (ascending, from 0), a tie to the one with the even index; larger values to the last."""
    mid = (grid[1:] + grid[:-1]) / 2
    odd = torch.arange(mid.numel(), device=mid.device) % 2 == 1
    return grid[torch.bucketize(a, mid[~odd], right=False) + torch.bucketize(a, mid[odd], right=True)]


def _encoded64(x, acts):
    dev = x.device
    if acts == "mxfp4":
        grid, top = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev), 2
    else:
        i = torch.arange(127, dtype=torch.float64, device=dev)
        grid, top = torch.where(i < 8, i * 2.0 ** -9, (1 + i % 8 / 8) * 2.0 ** (torch.floor(i / 8) - 7)), 8
    b = x.double().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1.0 - top, torch.full_like(amax, -127.0)).clamp(min=-127.0)
    return (torch.sign(b) * _nearest(b.abs() * 2.0 ** -e, grid) * 2.0 ** e).reshape(x.shape)


def _decoded64(buf, rows, k):
    v, s = _unpacked(buf, rows, k)
    return (v.double().reshape(*v.shape[:-1], -1, 32) * 2.0 ** (s.double() - 127)[..., None]).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode":
        w = _encoded64(s["w"], "mxfp4")
        return {"values": w, "looked_up": w[s["ids"].long()]}
    if op == "product":
        return _encoded64(s["x"], s["acts"]) @ _decoded64(s["w"], s["rows"], s["k"]).T
    n, top = s["ids"].shape
    ids = s["ids"].reshape(-1).tolist()
    lists = [[i for i, e in enumerate(ids) if e == j] for j in range(case["experts"])]
    order = [i for rows in lists for i in rows]
    kept = len(order)
    place = {slot: r for r, slot in enumerate(order)}
    slots = torch.tensor(order, dtype=torch.long, device=DEV)
    if op == "experts":
        x, out, at = _encoded64(s["x"], s["acts"]), torch.zeros((n * top, s["rows"]), dtype=torch.float64, device=DEV), 0
        for j, rows in enumerate(lists):
            if rows:
                out[at:at + len(rows)] = x[slots[at:at + len(rows)] // top] @ _decoded64(s["w"][j], s["rows"], s["k"]).T
                at += len(rows)
        return {"first": None, "row": None, "out": out}
    zero = torch.zeros(1, s["k"], dtype=torch.float64, device=DEV)
    x, answers = s["x"].double(), torch.cat((s["rows"].double()[:kept], zero))
    at = torch.tensor([place.get(i, kept) for i in range(n * top)], device=DEV).reshape(n, top)
    w, pad = s["weights"].double(), torch.zeros(n * top - kept, s["k"], dtype=torch.float64, device=DEV)
    out = {"first": None, "row": None, "sorted": torch.cat((x[slots // top], pad)), "y": torch.einsum("tj,tjk->tk", w, answers[at])}
    if case["train"]:
        dy, din = s["dy"].double(), torch.cat((s["dsorted"].double()[:kept], zero))
        out["drows"] = torch.cat((w.reshape(-1)[slots, None] * dy[slots // top], pad))
        out["dweights"] = torch.einsum("tk,tjk->tj", dy, answers[at])
        out["dx"] = din[at].sum(1)
    return out
