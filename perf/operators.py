"""Measured cases of the 4-bit key/value cache operators: kv4_append, kv4_read and kv4_attention.

The operators work on a paged cache of one attention layer, ``data`` uint8 [pages, heads, page/32,
tile bytes]. A tile holds 32 tokens of one head, keys and values of D coordinates each, as int4 codes
-7..7 in groups of G coordinates with one binary16 scale per group (value = code * scale), in an order
that the attention reads without shuffling (NG = D/G, little-endian 32-bit words of 8 codes, low nibble
first):

    keys          [32 tokens][4 c][D/32 j][8 i]                        coordinate 32 j + 8 c + i
    values        [2 s][2 h][8 r][4 c][2 b][D/32 j][4 i]               token 16 s + 8 h + 2 c + b,
                                                                       coordinate 32 j + 4 r + i
    key scales    [32 tokens][NG]
    value scales  [16 pairs][NG][2 b]                                  token 2 pair + b

``table`` [sequences, pages of a sequence] names each sequence's pages, ``lens`` its length after this
step and ``cu`` the offsets of its new tokens in the packed rows: new token i of n of a sequence of
length L stands at position L - n + i. With a rotation, keys and values are stored as T k and T v (T the
signed Walsh-Hadamard transform of size D over sqrt(D)); the attention rotates its queries by T and its
output back by its transpose.

  append     rotates, quantises and writes the new tokens, then reads the new rows back
  read       reads whole sequences back, in the original basis where the cache is rotated
  attention  softmax(q k / sqrt(D)) v over the cache; causal, with an optional window
"""
import math
import random

import numpy as np
import torch

own = False


def _case(name, op, batch, new, length, ragged, heads, share, dim, group, rotate, float32, window=0, page=64):
    return {"name": name, "op": op, "batch": batch, "new": new, "length": length, "ragged": ragged, "heads": heads,
            "share": share, "dim": dim, "group": group, "rotate": rotate, "float32": float32, "window": window,
            "page": page}


def listed():
    return [
        # one user's decoding step of a small model: 8 heads of 64, latency alone
        _case("append one token", "append", 1, 1, 700, False, 8, 4, 64, 32, True, False),
        # a serving batch's decoding step, float32 keys and values, one scale per row
        _case("append a batch's tokens", "append", 48, 1, 4000, True, 8, 4, 128, 128, True, True, page=32),
        # prompts of uneven lengths written in one call
        _case("append prompts", "append", 5, 3500, 3500, True, 8, 4, 128, 32, True, False),
        # a short odd cache handed to another kernel in float32, stored unrotated
        _case("read short, float32", "read", 3, 333, 333, True, 2, 8, 256, 64, False, True, page=128),
        # long sequences moved back to 16 bits, in the original basis
        _case("read long", "read", 6, 16001, 16001, True, 8, 4, 128, 32, True, False, page=256),
        # one user's decoding step at a short context of a small model: latency alone
        _case("decode short", "attention", 1, 1, 129, False, 8, 4, 64, 32, True, False),
        # one user at a very long context: the split over the length
        _case("decode long", "attention", 1, 1, 131000, False, 8, 4, 128, 32, True, False),
        # a serving batch at uneven contexts, shared heads
        _case("decode batch", "attention", 64, 1, 8192, True, 8, 4, 128, 32, True, False),
        # a serving batch with a key head for every query head (32 heads of 128) and one scale per row
        _case("decode unshared heads", "attention", 16, 1, 2048, True, 32, 1, 128, 128, True, False, page=32),
        # wide heads, many query heads on each key head, float32 queries, stored unrotated
        _case("decode wide heads", "attention", 4, 1, 5000, True, 2, 10, 256, 64, False, True),
        # drafted tokens verified together, with a sliding window
        _case("verify drafts in a window", "attention", 24, 6, 6000, True, 4, 8, 128, 64, True, False, window=1024),
        # the next chunk of two prompts over what the cache holds of them
        _case("chunk of a prompt", "attention", 2, 1024, 8192, True, 8, 4, 128, 32, True, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention"])
    dim = rng.choice([64, 128, 128, 256])
    c = {"op": op, "dim": dim, "group": rng.choice([g for g in (32, 64, 128, 256) if g <= dim]),
         "rotate": rng.random() < 0.7, "float32": rng.random() < 0.3, "page": rng.choice([32, 64, 128, 256]),
         "heads": rng.choice([1, 2, 4, 8, 32]), "share": rng.choice([1, 2, 4, 5, 8, 16]), "ragged": rng.random() < 0.8,
         "window": 0}
    room = 2 ** 28 // (c["heads"] * dim)  # tokens of the batch that stay below the largest listed case
    if op == "attention":
        c["new"] = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 700)])
        c["batch"] = _log(rng, 1, 64 if c["new"] < 9 else 4)
        top = room // c["batch"]
        if c["new"] >= 9:
            c["share"] = min(c["share"], 32 // min(32, c["heads"]) if c["heads"] > 1 else 8)
            top = min(top, 8192)
        c["length"] = min(max(_log(rng, 1, 100000), c["new"]), max(c["new"], top))
        c["window"] = _log(rng, 64, 2000) if rng.random() < 0.2 else 0
        most = 4.4e10 / (dim * c["batch"] * c["new"] * c["heads"] * c["share"])  # products of queries and keys
        c["new"] = min(c["new"], max(1, int(math.sqrt(most * c["new"]))))
        c["length"] = max(c["new"], min(c["length"], int(most)))
    else:
        c["batch"] = _log(rng, 1, 64)
        c["length"] = max(1, min(_log(rng, 1, 16000), room // (11 * c["batch"])))
        c["new"] = c["length"] if op == "read" else rng.choice([1, min(7, c["length"]), c["length"]])
    return c


def _lengths(case):
    """Lengths and new tokens of each sequence: the case's alone, so that work() knows them."""
    r = random.Random(case["batch"] * 7 + case["length"] * 3 + case["new"])
    lens, new = [case["length"]], [case["new"]]
    for _ in range(case["batch"] - 1):
        n = case["length"] if not case["ragged"] else r.randint(max(1, case["length"] // 4), case["length"])
        k = min(n, case["new"] if not case["ragged"] or case["new"] == 1 else r.randint(0, case["new"]))
        lens.append(n)
        new.append(n if case["op"] == "read" else k)
    return lens, new


def _tile_bytes(dim, group):
    return 32 * dim + 128 * dim // group


def _quantise(y, group):
    """Symmetric absmax codes and binary16 scales of float32 rows [..., D]: the decisions are taken in
    float32 on the stored scale, halves round away from zero, a scale that is zero or infinite gives 0."""
    g = y.unflatten(-1, (-1, group))
    s = (g.abs().amax(-1) / 7.0).to(torch.float16)
    s32 = s.float()[..., None]
    v = torch.where((s32 > 0) & torch.isfinite(s32), g / s32, torch.zeros_like(g))
    code = (v.sign() * (v.abs() + 0.5).floor()).clamp(-7, 7).to(torch.int8).flatten(-2)
    return code, s


def _nibbles(code):
    """int8 codes [..., n] packed two to a byte, low nibble first."""
    u = (code & 15).to(torch.uint8).unflatten(-1, (-1, 2))
    return u[..., 0] | (u[..., 1] << 4)


def _codes(packed):
    """The codes of packed bytes [..., n] as int8 [..., 2n]."""
    b = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).to(torch.int8)
    return (b ^ 8) - 8


def _pack_tiles(kc, ks, vc, vs):
    """Tiles [..., tile bytes] of codes [..., 32, D] and scales [..., 32, NG]."""
    lead, dim, ng = kc.shape[:-2], kc.shape[-1], ks.shape[-1]
    n = len(lead)
    at = list(range(n))
    k = kc.reshape(*lead, 32, dim // 32, 4, 8).transpose(-3, -2).reshape(*lead, 32 * dim)
    v = vc.reshape(*lead, 2, 2, 4, 2, dim // 32, 8, 4).permute(*at, n, n + 1, n + 5, n + 2, n + 3, n + 4, n + 6)
    v = v.reshape(*lead, 32 * dim)
    w = vs.reshape(*lead, 16, 2, ng).transpose(-2, -1).reshape(*lead, 32 * ng)
    return torch.cat((_nibbles(k), _nibbles(v), ks.reshape(*lead, 32 * ng).contiguous().view(torch.uint8),
                      w.contiguous().view(torch.uint8)), -1)


def _unpack_tiles(tiles, dim, ng):
    """Codes int8 [..., 32, D] and scales float16 [..., 32, NG] of keys and values."""
    lead = tiles.shape[:-1]
    n = len(lead)
    at = list(range(n))
    k = _codes(tiles[..., :16 * dim]).reshape(*lead, 32, 4, dim // 32, 8).transpose(-3, -2).reshape(*lead, 32, dim)
    v = _codes(tiles[..., 16 * dim:32 * dim]).reshape(*lead, 2, 2, 8, 4, 2, dim // 32, 4)
    v = v.permute(*at, n, n + 1, n + 3, n + 4, n + 5, n + 2, n + 6).reshape(*lead, 32, dim)
    s = tiles[..., 32 * dim:].contiguous().view(torch.float16)
    ks = s[..., :32 * ng].reshape(*lead, 32, ng)
    vs = s[..., 32 * ng:].reshape(*lead, 16, ng, 2).transpose(-2, -1).reshape(*lead, 32, ng)
    return k, ks, v, vs


def _hadamard(dim, dtype, device):
    """The Walsh-Hadamard matrix over sqrt(D): entry (r, c) has the sign (-1)^popcount(r & c)."""
    i = torch.arange(dim, device=device)
    both = i[:, None] & i[None, :]
    bits = (both[..., None] >> torch.arange(9, device=device)) & 1
    return (1 - 2 * (bits.sum(-1) & 1)).to(dtype) / math.sqrt(dim)


def prepare(case, seed):
    lens, new = _lengths(case)
    dim, heads, page, batch = case["dim"], case["heads"], case["page"], case["batch"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    per = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    own_pages = torch.tensor([-(-n // page) for n in lens], device="cuda")
    slot = torch.arange(per, device="cuda")[None, :]
    first = torch.cumsum(own_pages, 0) - own_pages
    table = torch.where(slot < own_pages[:, None], order[(first[:, None] + slot).clamp(max=pages - 1)], 0)
    signs = (1 - 2 * torch.randint(0, 2, (dim,), generator=g, device="cuda")).to(torch.int8)
    total = sum(new)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    state = {"case": case, "table": table.to(torch.int32).contiguous(), "signs": signs if case["rotate"] else None,
             "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "cu": cu, "total": total,
             "max_new": max(new), "max_len": max(lens)}
    kind = torch.float32 if case["float32"] else torch.bfloat16
    tiles, tb = page // 32, _tile_bytes(dim, case["group"])
    # pages as an allocator leaves them: whatever stood there before, infinities and NaN among the scales
    data = torch.randint(0, 256, (pages, heads, tiles, tb), generator=g, device="cuda", dtype=torch.uint8)
    if case["op"] != "append":
        # in the rotated basis keys and values are nearly normal; the values' mean is not zero
        step = max(1, 2 ** 27 // (heads * page * dim))
        tok = torch.arange(page, device="cuda").reshape(tiles, 32)
        left = torch.zeros(pages, dtype=torch.int64, device="cuda")  # valid tokens of each page
        held = (state["lens"][:, None] - slot * page).clamp(0, page)
        left[table[slot < own_pages[:, None]].long()] = held[slot < own_pages[:, None]].long()
        for a in range(0, pages, step):
            b = min(pages, a + step)
            kc, ks = _quantise(normal(b - a, heads, tiles, 32, dim), case["group"])
            vc, vs = _quantise(normal(b - a, heads, tiles, 32, dim) + 0.25, case["group"])
            stale = (tok[None] >= left[a:b, None, None])[:, None, :, :, None]
            old = _unpack_tiles(data[a:b], dim, dim // case["group"])
            data[a:b] = _pack_tiles(*[torch.where(stale, o, x) for o, x in zip(old, (kc, ks, vc, vs))])
    state["data"] = data
    if case["op"] == "append":
        hot = torch.where(torch.rand(dim, generator=g, device="cuda") < 0.02, 20.0, 1.0)  # outlier channels
        state["k"] = (normal(total, heads, dim) * hot).to(kind)
        state["v"] = normal(total, heads, dim).to(kind)
    elif case["op"] == "attention":
        state["q"] = (1.5 * normal(total, heads * case["share"], dim)).to(kind)
    if own:  # what a program keeps beside the cache's memory: its plan and the cache's handle
        import hadamard_butterfly_rotation_b200 as hbr
        plan = hbr.Plan.rht(dim, signs.cpu().numpy()) if case["rotate"] else None
        state["cache"] = hbr.KV4Cache(data, dim, case["group"], k_plan=plan, v_plan=plan)
    return state


def _owner(state):
    """The sequence and the position of every new token."""
    cu = state["cu"].long()
    t = torch.arange(state["total"], device="cuda")
    seq = torch.bucketize(t, cu[1:].contiguous(), right=True)
    return seq, state["lens"].long()[seq] - (cu[1:] - cu[:-1])[seq] + t - cu[:-1][seq]


def _places(state):
    """Byte offsets into the cache of each new token: packed keys, packed values, both scales."""
    c = state["case"]
    dim, ng = c["dim"], c["dim"] // c["group"]
    seq, pos = _owner(state)
    where = state["table"].long()[seq, pos // c["page"]]
    tile, t = pos % c["page"] // 32, (pos % 32)[:, None, None]
    head = torch.arange(c["heads"], device="cuda")
    tiles, tb = c["page"] // 32, _tile_bytes(dim, c["group"])
    base = (((where * c["heads"])[:, None] + head) * tiles + tile[:, None])[..., None] * tb
    byte = torch.arange(dim // 2, device="cuda")
    r, rest = byte // (dim // 16), byte % (dim // 16)
    k = base + t * (dim // 2) + byte
    v = base + 16 * dim + t // 8 * (4 * dim) + r * (dim // 2) + t % 8 // 2 * (dim // 8) + t % 2 * (dim // 16) + rest
    two = torch.arange(2 * ng, device="cuda")
    ks = base + 32 * dim + t * (2 * ng) + two
    vs = base + 32 * dim + 64 * ng + t // 2 * (4 * ng) + two // 2 * 4 + t % 2 * 2 + two % 2
    return k, v, ks, vs


def _rows_order(code, dim, values):
    """Codes [..., D] in the order of a cached row: keys [c][j][i], values [r][j][i]."""
    shape = (dim // 32, 8, 4) if values else (dim // 32, 4, 8)
    return code.unflatten(-1, shape).transpose(-3, -2).flatten(-3)


def _natural(code, dim, values):
    shape = (8, dim // 32, 4) if values else (4, dim // 32, 8)
    return code.unflatten(-1, shape).transpose(-3, -2).flatten(-3)


def _times(code, s, group):
    return (code.float().unflatten(-1, (-1, group)) * s.float()[..., None]).flatten(-2)


def _append(state):
    c = state["case"]
    dim, flat = c["dim"], state["data"].view(-1)
    k_at, v_at, ks_at, vs_at = _places(state)
    rows = torch.stack((state["k"], state["v"])).double()  # codes next to a border: the rotation in 64 bits
    if state["signs"] is not None:
        rows = (rows * state["signs"]) @ _hadamard(dim, torch.float64, "cuda")
    code, s = _quantise(rows.float(), c["group"])
    flat[k_at] = _nibbles(_rows_order(code[0], dim, False))
    flat[v_at] = _nibbles(_rows_order(code[1], dim, True))
    flat[ks_at] = s[0].contiguous().view(torch.uint8)
    flat[vs_at] = s[1].contiguous().view(torch.uint8)
    k = _times(_natural(_codes(flat[k_at]), dim, False), flat[ks_at].view(torch.float16), c["group"])
    v = _times(_natural(_codes(flat[v_at]), dim, True), flat[vs_at].view(torch.float16), c["group"])
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _dense(state):
    """Keys and values of every sequence up to the longest, float32 [sequences, tokens, heads, D], and which are real."""
    c = state["case"]
    dim, ng = c["dim"], c["dim"] // c["group"]
    tiles = state["data"][state["table"].long()].permute(0, 1, 3, 2, 4).flatten(1, 2)  # [B, tiles, heads, bytes]
    kc, ks, vc, vs = _unpack_tiles(tiles, dim, ng)
    real = torch.arange(tiles.shape[1] * 32, device="cuda")[None] < state["lens"][:, None]
    mask = real.unflatten(1, (-1, 32))[:, :, None, :, None]
    zero = torch.zeros((), dtype=torch.float16, device="cuda")
    k = _times(kc, torch.where(mask, ks, zero), c["group"]).transpose(2, 3).flatten(1, 2)
    v = _times(vc, torch.where(mask, vs, zero), c["group"]).transpose(2, 3).flatten(1, 2)
    return k, v, real


def _back(state, x):
    """From the cache's basis to the original one."""
    return x if state["signs"] is None else (x @ _hadamard(x.shape[-1], x.dtype, "cuda")) * state["signs"]


def _read(state):
    k, v, _ = _dense(state)
    at = _owner(state)
    kind = torch.float32 if state["case"]["float32"] else torch.bfloat16
    return _back(state, k[at]).to(kind), _back(state, v[at]).to(kind)


def _attention(state):
    c = state["case"]
    dim, share, heads = c["dim"], c["share"], c["heads"]
    k, v, real = _dense(state)
    seq, pos = _owner(state)
    row = torch.arange(state["total"], device="cuda") - state["cu"].long()[seq]
    q = state["q"].float()
    if state["signs"] is not None:
        q = (q * state["signs"]) @ _hadamard(dim, torch.float32, "cuda")
    rows = torch.zeros(c["batch"], state["max_new"], heads * share, dim, device="cuda")
    at = torch.full((c["batch"], state["max_new"]), -1, device="cuda")
    rows[seq, row], at[seq, row] = q, pos
    rows = rows.reshape(c["batch"], -1, heads, share, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    logit = rows @ k.permute(0, 2, 3, 1) / math.sqrt(dim)  # [B, heads, new * share, tokens]
    key = torch.arange(k.shape[1], device="cuda")
    seen = (key <= at[..., None]) & real[:, None]
    if c["window"]:
        seen &= key > at[..., None] - c["window"]
    logit = logit.unflatten(2, (-1, share)).masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    o = (p @ v.transpose(1, 2)) / p.sum(-1, keepdim=True).clamp(min=1e-38)
    o = o.unflatten(2, (-1, share)).transpose(1, 2)[seq, row].flatten(1, 2)
    return _back(state, o).to(torch.bfloat16)


def run(state):
    c = state["case"]
    if own:
        import hadamard_butterfly_rotation_b200 as hbr
        where = (state["cache"], state["table"], state["lens"], state["cu"])
        if c["op"] == "append":
            hbr.kv4_append(where[0], state["k"], state["v"], *where[1:])
            return hbr.kv4_read(*where, total=state["total"], out_dtype=torch.bfloat16)
        if c["op"] == "read":
            kind = torch.float32 if c["float32"] else torch.bfloat16
            return hbr.kv4_read(*where, total=state["total"], inverse=c["rotate"], out_dtype=kind)
        return hbr.kv4_attention(state["q"], *where, max_new=state["max_new"], max_len=state["max_len"],
                                 window=c["window"])
    return {"append": _append, "read": _read, "attention": _attention}[c["op"]](state)


def work(case):
    lens, new = _lengths(case)
    dim, heads, window = case["dim"], case["heads"], case["window"]
    token = heads * (dim + 4 * dim // case["group"])  # cached bytes of a token, keys and values
    item = 4 if case["float32"] else 2
    if case["op"] == "append":  # rows in, cache out, rows back in bf16
        n = sum(new)
        return {"bytes": n * (2 * heads * dim * (item + 2) + token), "flops": n * 2 * heads * dim * (math.log2(dim) + 3)}
    if case["op"] == "read":
        n = sum(new)
        return {"bytes": n * (2 * heads * dim * item + token), "flops": n * 2 * heads * dim * (math.log2(dim) + 1)}
    held = pairs = 0
    for n, k in zip(lens, new):
        low = n - k  # the first new token's position
        held += 0 if not k else n - (max(0, low + 1 - window) if window else 0)
        pairs += sum(min(low + i + 1, window) if window else low + i + 1 for i in range(k))
    rows = sum(new) * heads * case["share"]
    return {"bytes": held * token + rows * dim * (item + 2), "flops": 4.0 * dim * heads * case["share"] * pairs}


def _cached(state, b, n):
    """Keys and values of the first n tokens of one sequence in 64 bits [n, heads, D], code by code."""
    c = state["case"]
    dim, ng = c["dim"], c["dim"] // c["group"]
    t = torch.arange(n, device="cuda")
    page = state["data"][state["table"][b, t // c["page"]].long(), :, (t % c["page"]) // 32]  # [n, heads, bytes]
    t = (t % 32)[:, None]
    d = torch.arange(dim, device="cuda")[None]
    grp = torch.arange(ng, device="cuda")[None]
    k_nib = t * dim + d // 8 % 4 * (dim // 4) + d // 32 * 8 + d % 8
    v_nib = ((t // 8 * 8 + d % 32 // 4) * 4 + t % 8 // 2) * (dim // 4) + t % 2 * (dim // 8) + d // 32 * 4 + d % 4
    k_s, v_s = t * ng + grp, (t // 2 * ng + grp) * 2 + t % 2 + 32 * ng
    out = []
    for nib, sc in ((k_nib, k_s), (v_nib + 32 * dim, v_s)):
        byte = torch.gather(page, 2, (nib // 2)[:, None].expand(-1, c["heads"], -1))
        code = torch.where(nib[:, None] % 2 == 1, byte >> 4, byte & 15).double()
        code = torch.where(code > 7, code - 16, code)
        two = torch.stack((sc * 2, sc * 2 + 1), -1).flatten(1) + 32 * dim
        s = torch.gather(page, 2, two[:, None].expand(-1, c["heads"], -1)).contiguous().view(torch.float16).double()
        out.append(code * s.repeat_interleave(c["group"], -1))
    return out


def _butterfly(x):
    """The Walsh-Hadamard transform over sqrt(D) of the last axis, by halves."""
    dim, h = x.shape[-1], 1
    while h < dim:
        a, b = x.unflatten(-1, (-1, 2, h)).unbind(-2)
        x = torch.stack((a + b, a - b), -2).flatten(-3)
        h *= 2
    return x / math.sqrt(dim)


def exact(case, seed):
    state = prepare(case, seed)
    lens, new = _lengths(case)
    signs, dim, share = state["signs"], case["dim"], case["share"]
    if case["op"] == "append":
        both = []
        for x in (state["k"].double(), state["v"].double()):
            y = (x if signs is None else _butterfly(x * signs.double())).unflatten(-1, (-1, case["group"]))
            s = (y.abs().amax(-1, keepdim=True) / 7).to(torch.float16).double()
            v = torch.where(s > 0, y / s, 0.0 * y)
            both.append(((v.abs() + 0.5).floor().clamp(max=7) * v.sign() * s).flatten(-2))
        return tuple(both)
    both, outs, first = ([], []), [], 0
    for b in range(case["batch"]):
        n, m = lens[b], new[b]
        if m == 0:
            continue
        k, v = _cached(state, b, n)
        if case["op"] == "read":
            for x, to in zip((k, v), both):
                to.append(x if signs is None else _butterfly(x) * signs.double())
            continue
        q = state["q"][first:first + m].double()
        first += m
        if signs is not None:
            q = _butterfly(q * signs.double())
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        shut = (key > pos) | ((key <= pos - case["window"]) if case["window"] else False)
        o = torch.empty_like(q)
        for h in range(case["heads"] * share):
            z = (q[:, h] @ k[:, h // share].T / math.sqrt(dim)).masked_fill(shut, -math.inf)
            o[:, h] = torch.softmax(z, -1) @ v[:, h // share]
        outs.append(o if signs is None else _butterfly(o) * signs.double())
    return torch.cat(outs) if case["op"] == "attention" else tuple(torch.cat(x) for x in both)
