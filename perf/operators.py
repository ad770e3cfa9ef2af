"""The paged 4-bit KV cache: tokens quantised as they are written, read back, and attended to (with a sliding window and
sinks, from one query token per sequence to a prefill chunk).  Workloads and plain forms.

The cache ("pool") is one byte buffer [page][kv head][16-token tile][tile bytes].  A tile of 16 tokens of one KV head holds, for
G = d / 32 groups of 32 head-dim elements: the key codes [G][16 tokens][16 bytes] (element e of a group in nibble e), the value
codes likewise, the keys' fp16 step and offset [16 tokens][G][s, m] and the values' [8 token pairs][G][s, s', m, m'].
A group's grid: s = fp16((max - min) / 15), m = fp16(min), code = clamp(floor((w - m) / s + 1/2), 0, 15), value m + s code.
Token slot = page * page_size + place in the page.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
LIMIT = 65408.0  # values are clamped to this before they are quantised


def listed():
    return [
        # the new token of one decode step, from the fp32 qkv projection row: latency
        {"name": "write_decode_1_fp32", "op": "write", "n": 1, "h_q": 32, "h_kv": 8, "d": 128, "page": 16, "dtype": "fp32"},
        # the new tokens of a batch of sequences, each in a page of its own
        {"name": "write_decode_61_fp16", "op": "write", "n": 61, "h_q": 16, "h_kv": 4, "d": 64, "page": 32, "dtype": "fp16"},
        # a prefill chunk
        {"name": "write_prefill_8192_bf16", "op": "write", "n": 8192, "h_q": 32, "h_kv": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # a handful of sequences read back (a cache that moves to another format), odd total
        {"name": "read_5003_fp16", "op": "read", "n": 5003, "h_kv": 8, "d": 128, "page": 16, "dtype": "fp16"},
        # a whole long context read back
        {"name": "read_131072_bf16", "op": "read", "n": 131072, "h_kv": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # single-token attention at the context lengths the framework serves
        {"name": "decode_8192_fp16", "op": "attend", "batch": 1, "nq": 1, "len": 8192, "ragged": False, "h_q": 32, "h_kv": 8, "d": 128,
         "page": 16, "window": 0, "sinks": 0, "dtype": "fp16"},
        {"name": "decode_131072_fp16", "op": "attend", "batch": 1, "nq": 1, "len": 131072, "ragged": False, "h_q": 32, "h_kv": 8, "d": 128,
         "page": 64, "window": 0, "sinks": 0, "dtype": "fp16"},
        {"name": "decode_8x32769_bf16", "op": "attend", "batch": 8, "nq": 1, "len": 32769, "ragged": False, "h_q": 32, "h_kv": 8, "d": 128,
         "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a server's batch: lengths from one token up, sliding window with sinks
        {"name": "decode_64_window_fp16", "op": "attend", "batch": 64, "nq": 1, "len": 8191, "ragged": True, "h_q": 32, "h_kv": 8, "d": 128,
         "page": 32, "window": 1024, "sinks": 4, "dtype": "fp16"},
        # drafted tokens checked: a few query tokens per sequence
        {"name": "verify_16x5_bf16", "op": "attend", "batch": 16, "nq": 5, "len": 4099, "ragged": True, "h_q": 16, "h_kv": 4, "d": 64,
         "page": 16, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a prefill chunk behind a long prefix
        {"name": "prefill_2048_at_16384_bf16", "op": "attend", "batch": 1, "nq": 2048, "len": 16384, "ragged": False, "h_q": 32, "h_kv": 8,
         "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # whole prompts under a sliding window with sinks, odd lengths
        {"name": "prefill_2x4001_window_fp16", "op": "attend", "batch": 2, "nq": 4001, "len": 4001, "ragged": True, "h_q": 32, "h_kv": 8,
         "d": 128, "page": 16, "window": 1024, "sinks": 4, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d, h_kv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    page, op = rng.choice([16, 32, 64, 128, 256]), rng.choice(["write", "read", "attend", "attend", "attend"])
    case = {"op": op, "h_kv": h_kv, "d": d, "page": page}
    if op == "write":
        return case | {"n": _log(rng, 1, 8192), "h_q": h_kv * group, "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    if op == "read":
        dtype = rng.choice(["fp16", "bf16", "fp32"])
        return case | {"n": _log(rng, 1, 131072 if dtype != "fp32" else 65536), "dtype": dtype}
    kind = rng.choice(["decode", "decode", "verify", "prefill"])
    if kind == "decode":
        batch = _log(rng, 1, 64)
        nq, length = 1, _log(rng, 1, 262144 // batch if batch > 2 else 131072)
    elif kind == "verify":
        batch, nq = _log(rng, 1, 32), rng.randint(2, 8)
        length = _log(rng, nq, 4096)
    else:
        batch, nq = rng.choice([1, 1, 2, 3]), _log(rng, 9, 4096)
        length = min(16384, nq + rng.choice([0, _log(rng, 1, 8192)]))
        while batch * nq * length * h_kv * group * d > 2048 * 16384 * 32 * 128:
            batch, nq, length = max(1, batch - 1), max(9, nq // 2), max(9, length // 2)
        length = max(length, nq)
    return case | {"batch": batch, "nq": nq, "len": length, "ragged": batch > 1 and rng.random() < 0.7, "h_q": h_kv * group,
                   "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "sinks": rng.choice([0, 4, _log(rng, 1, 100)]),
                   "dtype": rng.choice(["fp16", "bf16"])}


def _lengths(case):
    """Cached tokens and query tokens of each sequence (part of the workload, known on the host)."""
    b = case["batch"]
    if not case["ragged"]:
        return [case["len"]] * b, [case["nq"]] * b
    # spread from one token (or the queries alone) to the full length; query counts from one to all
    q = [max(1, round(case["nq"] * (i + 1) / b)) if case["nq"] > 8 else case["nq"] for i in range(b)]
    return [max(q[i], round(case["len"] * ((i * 37) % b + 1) / b)) for i in range(b)], q


def _tile_bytes(d):
    return 16 * (d + d // 4)


def _sections(pool, case):
    """Views of the pool's parts: key codes, value codes [page][head][tile][G][16][16], key grid [..][16][G][2], value grid [..][8][G][2][2]."""
    h, d, page = case["h_kv"], case["d"], case["page"]
    g = d // 32
    t = pool.view(-1, h, page // 16, _tile_bytes(d))
    kc = t[..., : 8 * d].unflatten(-1, (g, 16, 16))
    vc = t[..., 8 * d : 16 * d].unflatten(-1, (g, 16, 16))
    ks = t[..., 16 * d : 18 * d].view(torch.float16).unflatten(-1, (16, g, 2))
    vs = t[..., 18 * d :].view(torch.float16).unflatten(-1, (8, g, 2, 2))
    return kc, vc, ks, vs


def _place(slots, page):
    s = slots.long()
    return s // page, s % page // 16, s % 16


def _grid(x):
    """Codes (one per element), step and offset of x [..][d]: decided in 64 bits, as values next to a border have to be."""
    w = torch.where(torch.isnan(x), torch.zeros((), dtype=x.dtype, device=x.device), x).double().clamp(-LIMIT, LIMIT).unflatten(-1, (-1, 32))
    lo, hi = w.amin(-1), w.amax(-1)
    s, m = ((hi - lo) / 15).to(torch.float16), lo.to(torch.float16)
    sd, md = s.double()[..., None], m.double()[..., None]
    q = torch.floor((w - md) / torch.where(sd == 0, torch.ones_like(sd), sd) + 0.5).clamp(0, 15)
    return torch.where(sd == 0, torch.zeros_like(q), q).to(torch.uint8), s, m


def _store(pool, case, k, v, slots):
    kc, vc, ks, vs = _sections(pool, case)
    p, u, t = _place(slots, case["page"])
    for x, codes, is_value in ((k, kc, False), (v, vc, True)):
        q, s, m = _grid(x)
        codes[p, :, u, :, t] = q[..., 0::2] | (q[..., 1::2] << 4)
        if is_value:
            vs[p, :, u, t // 2, :, 0, t % 2] = s
            vs[p, :, u, t // 2, :, 1, t % 2] = m
        else:
            ks[p, :, u, t] = torch.stack((s, m), -1)


def _load(pool, case, slots):
    """Keys and values of the slots, fp32 [..][h_kv][d]."""
    kc, vc, ks, vs = _sections(pool, case)
    p, u, t = _place(slots, case["page"])
    wide = lambda c: torch.stack((c & 15, c >> 4), -1).flatten(-2).float()  # noqa: E731
    sm = ks[p, :, u, t].float()
    k = (sm[..., 1:] + sm[..., :1] * wide(kc[p, :, u, :, t])).flatten(-2)
    s, m = vs[p, :, u, t // 2, :, 0, t % 2].float(), vs[p, :, u, t // 2, :, 1, t % 2].float()
    return k, (m[..., None] + s[..., None] * wide(vc[p, :, u, :, t])).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    h, d, page, dtype = case["h_kv"], case["d"], case["page"], DTYPES[case["dtype"]]

    def keys_values(n):
        # keys with four large channels per head, as the framework's caches have them
        k, v = rand(n, h, d), rand(n, h, d)
        loud = torch.rand(h, d, device="cuda", generator=g).argsort(-1)[:, :4]
        k.scatter_(2, loud.expand(n, h, 4), k.gather(2, loud.expand(n, h, 4)) * 10)
        return k, v

    def pool_of(pages):
        return torch.zeros(pages * h * page // 16 * _tile_bytes(d), dtype=torch.uint8, device="cuda")

    def fill(pool, slots):
        for part in slots.split(32768):
            _store(pool, case, *(x.half() for x in keys_values(len(part))), part)

    if case["op"] == "write":
        n = case["n"]
        # a page each for single tokens of many sequences; whole pages for a chunk
        spread = n <= 64
        pages = n if spread else -(-n // page)
        table = torch.randperm(pages + 3, device="cuda", generator=g)[:pages]
        i = torch.arange(n, device="cuda")
        place = torch.randint(0, page, (n,), device="cuda", generator=g)
        slots = (table * page + place if spread else table[i // page] * page + i % page).int()
        qkv = rand(n, (case["h_q"] + 2 * h) * d)
        k, v = keys_values(n)
        a, b = case["h_q"] * d, (case["h_q"] + h) * d
        qkv[:, a:b], qkv[:, b:] = k.flatten(1), v.flatten(1)
        qkv = qkv.to(dtype)  # the projection's output: keys and values are views of it
        return {"case": case, "pool": pool_of(pages + 3), "k": qkv[:, a:b].unflatten(1, (h, d)), "v": qkv[:, b:].unflatten(1, (h, d)), "slots": slots}
    if case["op"] == "read":
        n = case["n"]
        pages = -(-n // page) + 3
        table = torch.randperm(pages, device="cuda", generator=g)
        i = torch.arange(n, device="cuda")
        slots = (table[i // page] * page + i % page).int()
        pool = pool_of(pages)
        fill(pool, slots)
        return {"case": case, "pool": pool, "slots": slots}
    lens, nqs = _lengths(case)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    order = torch.randperm(pages, device="cuda", generator=g)[: sum(counts)].int()
    table = torch.full((case["batch"], max(counts)), -1, dtype=torch.int32)
    at = 0
    slots = []
    order_h = order.cpu()
    for b, (c, n) in enumerate(zip(counts, lens)):
        table[b, :c] = order_h[at : at + c]
        at += c
        i = torch.arange(n)
        slots.append(table[b, i // page] * page + i % page)
    pool = pool_of(pages)
    fill(pool, torch.cat(slots).int().cuda())
    cu = [0]
    for n in nqs:
        cu.append(cu[-1] + n)
    return {"case": case, "pool": pool, "pages": table.cuda(), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "cu_q": torch.tensor(cu, dtype=torch.int32, device="cuda"), "q": rand(cu[-1], case["h_q"], d).to(dtype),
            "max_len": max(lens), "max_nq": max(nqs), "scale": d ** -0.5}


def _cache(state):
    """The handle that a program keeps with its pool."""
    if "cache" not in state:
        from bit_decode_selective_b200.ops import PagedKVCache

        case, pool = state["case"], state["pool"]
        per_page = case["h_kv"] * case["page"] // 16 * _tile_bytes(case["d"])
        state["cache"] = PagedKVCache(pool.numel() // per_page, case["page"], case["h_kv"], case["d"], pool=pool)
    return state["cache"]


def _attend(pool, case, q, pages, lens, cu_q, max_len, max_nq, scale):
    """Plain form: every sequence padded to the longest, 32 bits throughout."""
    page, h = case["page"], case["h_kv"]
    j = torch.arange(max_len, device=q.device)
    table = pages.long()[:, j // page].clamp(min=0)
    k, v = _load(pool, case, table * page + j % page)  # [B][L][h][d]
    nq = (cu_q[1:] - cu_q[:-1]).long()
    i = torch.arange(max_nq, device=q.device)
    rows = (cu_q[:-1].long()[:, None] + i).clamp(max=q.shape[0] - 1)
    x = q.float()[rows].unflatten(2, (h, -1))  # [B][nq][h][group][d]
    logits = torch.einsum("bihgd,bjhd->bhgij", x, k) * scale
    pos = (lens.long() - nq)[:, None] + i  # [B][nq]
    seen = j <= pos[..., None]
    if case["window"]:
        seen &= (j > pos[..., None] - case["window"]) | (j < case["sinks"])
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(logits - logits.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    out = torch.einsum("bhgij,bjhd->bihgd", p, v).flatten(2, 3).to(q.dtype)
    # back to the packed rows
    row = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu_q[1:].long(), row, right=True)
    return out[b, row - cu_q.long()[b]]


def run(state):
    case, pool = state["case"], state["pool"]
    if case["op"] == "write":
        if own:
            cache = _cache(state)
            cache.write(state["k"], state["v"], state["slots"])
            return cache.read(state["slots"], DTYPES[case["dtype"]])
        _store(pool, case, state["k"], state["v"], state["slots"])
        return tuple(x.to(DTYPES[case["dtype"]]) for x in _load(pool, case, state["slots"]))
    if case["op"] == "read":
        if own:
            return _cache(state).read(state["slots"], DTYPES[case["dtype"]])
        return tuple(x.to(DTYPES[case["dtype"]]) for x in _load(pool, case, state["slots"]))
    if own:
        cu_q = state["cu_q"] if case["nq"] > 1 else None
        return _cache(state).attend(state["q"], state["pages"], state["lens"], cu_q=cu_q, scale=state["scale"], window=case["window"],
                                    sinks=case["sinks"])
    return _attend(pool, case, state["q"], state["pages"], state["lens"], state["cu_q"], state["max_len"], state["max_nq"], state["scale"])


def _visible(case, lens, nqs):
    """Cached tokens that some query sees, and (query, token) pairs, over all sequences."""
    tokens = pairs = 0
    w, sinks = case["window"], case["sinks"]
    for n, c in zip(lens, nqs):
        if not w:
            tokens += n
            pairs += c * (n - c) + c * (c + 1) // 2
            continue
        lo = max(0, n - c - w + 1)
        tokens += n - lo + min(lo, sinks)
        for p in range(n - c, n):
            first = max(0, p - w + 1)
            pairs += p + 1 - first + min(first, sinks)
    return tokens, pairs


def work(case):
    h, d, e = case["h_kv"], case["d"], 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "write":  # values in, codes and grids out, the values they stand for out
        return {"bytes": case["n"] * h * (4 * d * e + d + d // 4) + 4 * case["n"], "flops": case["n"] * h * d * 2 * 10}
    if case["op"] == "read":
        return {"bytes": case["n"] * h * (2 * d * e + d + d // 4) + 4 * case["n"], "flops": case["n"] * h * d * 2 * 2}
    lens, nqs = _lengths(case)
    tokens, pairs = _visible(case, lens, nqs)
    return {"bytes": tokens * h * (d + d // 4) + 2 * sum(nqs) * case["h_q"] * d * e, "flops": 4 * d * case["h_q"] * pairs}


# ---- the definition in 64 bits ----------------------------------------------------------------------------------------------------


def _exact_value(x):
    """What a token's values [n][h][d] stand for once quantised."""
    n, h, d = x.shape
    w = x.double().nan_to_num(nan=0.0, posinf=LIMIT, neginf=-LIMIT).reshape(n, h, d // 32, 32)
    w = torch.minimum(torch.maximum(w, w.new_tensor(-LIMIT)), w.new_tensor(LIMIT))
    low = w.min(dim=3, keepdim=True).values
    step = ((w.max(dim=3, keepdim=True).values - low) / 15).half().double()
    offset = low.half().double()
    code = torch.floor((w - offset) / step + 0.5)
    code = torch.where(step > 0, code.clamp(0, 15), torch.zeros_like(code))
    return (offset + step * code).reshape(n, h, d)


def _exact_tokens(pool, case, slots):
    """fp64 keys and values [n][h][d] of host-known slots, read byte by byte from their addresses."""
    h, d, page = case["h_kv"], case["d"], case["page"]
    g, tile = d // 32, _tile_bytes(d)
    dev = pool.device
    s = slots.to(dev).long()
    base = ((s // page)[:, None] * h + torch.arange(h, device=dev)) * (page // 16) + (s % page // 16)[:, None]
    base = base * tile  # [n][h]
    t = (s % 16)[:, None, None]
    e = torch.arange(d, device=dev)
    byte = (e // 32) * 256 + (e % 32) // 2 + t * 16 + base[..., None]
    half = pool.view(torch.float16)
    out = []
    for value in (0, 1):
        code = (pool[byte + 8 * d * value].long() >> (4 * (e % 2))) & 15
        grp = e // 32
        if value:
            at = base[..., None] // 2 + 9 * d + (t // 2 * g + grp) * 4 + t % 2
            step, offset = half[at], half[at + 2]
        else:
            at = base[..., None] // 2 + 8 * d + (t * g + grp) * 2
            step, offset = half[at], half[at + 1]
        out.append(offset.double() + step.double() * code.double())
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "write":
        return _exact_value(state["k"]), _exact_value(state["v"])
    if case["op"] == "read":
        parts = [_exact_tokens(state["pool"], case, s) for s in state["slots"].split(16384)]
        return tuple(torch.cat([p[i] for p in parts]) for i in (0, 1))
    lens, nqs = _lengths(case)
    h, group, page = case["h_kv"], case["h_q"] // case["h_kv"], case["page"]
    rows, start = [], 0
    for b, (n, c) in enumerate(zip(lens, nqs)):
        j = torch.arange(n, device="cuda")
        slots = state["pages"][b].long()[j // page] * page + j % page
        parts = [_exact_tokens(state["pool"], case, s) for s in slots.split(16384)]
        k, v = (torch.cat([p[i] for p in parts]) for i in (0, 1))
        q = state["q"][start : start + c].double()
        start += c
        for q0 in range(0, c, 1024):
            x = q[q0 : q0 + 1024]
            p = n - c + q0 + torch.arange(x.shape[0], device="cuda")
            hidden = j[None, :] > p[:, None]
            if case["window"]:
                hidden |= (j[None, :] <= p[:, None] - case["window"]) & (j[None, :] >= case["sinks"])
            heads = []
            for hq in range(case["h_q"]):
                logit = (x[:, hq] @ k[:, hq // group].T) * state["scale"]
                heads.append(torch.softmax(logit.masked_fill(hidden, -math.inf), -1) @ v[:, hq // group])
            rows.append(torch.stack(heads, 1))
    return torch.cat(rows)
