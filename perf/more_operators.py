"""Measured cases of a 4-bit cache in pages and of int8 products: attention over cached keys and
values held in 4 bits, the write and read-back of that cache, the pages it lies in (forked, grown with
copies on write, compacted), and the matrix product of int8 tokens and int8 weights with a scale for each
token and channel.

``run`` computes a case in plain torch operations, or, with ``own`` set, through this
package's operators. Sizes are the package's 2B / 7B / 100B class layers (hidden 2560 / 4096 /
8192 with 20/5, 32/32 and 64/8 heads of 128, vocabulary 32000) and generic ones around them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
GROUP = 32  # values of a token and head that share a scale
TILE = 16  # tokens whose codes lie together


def listed():
    return [
        # One request's next token, 2B class: latency.
        {"name": "cache4 attention 1 token, 777 keys", "op": "attention", "q": "1", "k": "777", "heads": 20,
         "kv_heads": 5, "dim": 128, "page": 16, "type": "bf16", "out": "bf16", "causal": True},
        # A decode batch of long conversations filled to different lengths, one of them empty.
        {"name": "cache4 attention decode 64 x 8192", "op": "attention", "q": ",".join(["1"] * 64),
         "k": ",".join(str((i * 2654435761 + 97) % 8192 if i != 13 else 0) for i in range(63)) + ",8192",
         "heads": 20, "kv_heads": 5, "dim": 128, "page": 64, "type": "bf16", "out": "fp32", "causal": True},
        # Drafts of five tokens checked for sixteen requests of a 100B class model.
        {"name": "cache4 attention drafts 16 x 5", "op": "attention", "q": ",".join(["5"] * 16),
         "k": ",".join(str((i * 331 + 5) % 3000 + 5) for i in range(16)), "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 32, "type": "fp16", "out": "fp16", "causal": True},
        # Prompts continued behind cached keys, 7B class, packed with one decoding request.
        {"name": "cache4 attention continued prompts 7B", "op": "attention", "q": "512,1,300", "k": "4608,2049,300",
         "heads": 32, "kv_heads": 32, "dim": 128, "page": 64, "type": "bf16", "out": "bf16", "causal": True},
        # A decode batch's new keys and values into their pages, with padding tokens.
        {"name": "cache4 write 37 tokens 2B", "op": "write", "tokens": 37, "kv_heads": 5, "dim": 128, "page": 16,
         "pages": 12, "type": "bf16"},
        # A long prompt's keys and values, 100B class.
        {"name": "cache4 write 16384 tokens 100B", "op": "write", "tokens": 16384, "kv_heads": 8, "dim": 128,
         "page": 64, "pages": 300, "type": "fp16"},
        # One step of a beam search over a few beams: reorder, then a token each, last pages copied where shared.
        {"name": "pages beam step 8", "op": "step", "seqs": 8, "most": 9, "page": 32, "pages": 96, "layers": 30,
         "page_bytes": 21760, "new": 1, "ended": 0},
        # A serving step: some requests end, the others go on, new prompts come in.
        {"name": "pages serving step 256", "op": "step", "seqs": 256, "most": 64, "page": 16, "pages": 20000,
         "layers": 2, "page_bytes": 2720, "new": 300, "ended": 40},
        # A fragmented pool brought together, to hand the rest back.
        {"name": "pages compact 4096", "op": "compact", "seqs": 64, "most": 40, "page": 64, "pages": 4096,
         "layers": 4, "page_bytes": 43520},
        # The output head of a 2B class model for one token.
        {"name": "int8 head 1 token 2B", "op": "int8", "tokens": 1, "k": 2560, "n": 32000, "out": "fp32",
         "bias": False},
        # A ragged decode batch at a 7B class gate+up projection.
        {"name": "int8 37 requests 7B gate_up", "op": "int8", "tokens": 37, "k": 4096, "n": 22016, "out": "bf16",
         "bias": True},
        # Packed prompts at a 100B class gate projection.
        {"name": "int8 prompts 4096 100B", "op": "int8", "tokens": 4096, "k": 8192, "n": 28672, "out": "bf16",
         "bias": False},
    ]


HEADS = [(20, 5, 128), (32, 32, 128), (64, 8, 128), (16, 2, 64), (8, 1, 256), (6, 3, 80), (12, 4, 96)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "write", "step", "compact", "int8", "int8"])
    if op == "int8":
        tokens = _log(rng, 1, 4096)
        return {"op": "int8", "tokens": tokens, "k": _log(rng, 64, 11008), "n": _log(rng, 64, 24000),
                "out": rng.choice(["fp32", "bf16", "fp16"]), "bias": rng.random() < 0.4}
    if op in ("step", "compact"):
        seqs, most, page = _log(rng, 1, 300), _log(rng, 2, 64), rng.choice([16, 32, 64, 128])
        layers, page_bytes = _log(rng, 1, 32), 16 * _log(rng, 34, 2720)
        pages = max(8, min(seqs * (most + 2), 250000000 // (layers * page_bytes)))
        case = {"op": op, "seqs": seqs, "most": most, "page": page, "pages": pages, "layers": layers,
                "page_bytes": page_bytes}
        if op == "step":
            case.update(new=rng.choice([1, 1, 5, 200]), ended=rng.choice([0, 0, seqs // 4]))
        return case
    heads, kv_heads, dim = rng.choice(HEADS)
    if op == "write":
        tokens, page = _log(rng, 1, 12000), rng.choice([16, 32, 64, 128])
        return {"op": "write", "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page,
                "pages": tokens // page + rng.choice([1, 2, 17]), "type": rng.choice(["bf16", "fp16", "fp32"])}
    kind = rng.choice(["bf16", "bf16", "fp16"])
    case = {"op": "attention", "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": rng.choice([16, 32, 64, 128]), "type": kind, "out": rng.choice([kind, kind, "fp32"]),
            "causal": rng.random() < 0.85}
    if rng.random() < 0.7:  # decode, drafts of a few tokens, one of them a short prompt
        n, longest = _log(rng, 1, 96), _log(rng, 16, 6000)
        most = rng.choice([1, 1, 4, 33])
        q = [rng.randint(min(1, most - 1), most) for _ in range(n)]
        q[rng.randrange(n)] = most
        k = [rng.randint(0, longest) for _ in q]
    else:  # prompts, some behind cached keys
        q = [_log(rng, 1, 1000) for _ in range(rng.randint(1, 4))]
        k = [v + rng.choice([0, 0, rng.randint(1, 3000)]) for v in q]
    case.update(q=",".join(map(str, q)), k=",".join(map(str, k)))
    return case


def _ints(text):
    return [int(v) for v in text.split(",")]


def _i32(values):
    return torch.as_tensor(np.asarray(values, dtype=np.int32), device=DEV)


# ------------------------------------------------------- the 4-bit format, in torch


def _levels(dtype=torch.float32):
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-x for x in v], dtype=dtype, device=DEV)


def _encode(x):
    """(codes 0..15, scale bytes) of x [..., dim], groups of 32 along the last dimension (the last one filled
    with zeros): scale 2^e with the smallest e such that no value of the group is above 7 * 2^e."""
    wide = -(-x.shape[-1] // GROUP) * GROUP
    x = torch.nn.functional.pad(x.float(), (0, wide - x.shape[-1])).unflatten(-1, (-1, GROUP))
    most, e = torch.frexp(x.abs().amax(-1))  # most * 2^e, most in [0.5, 1)
    e = torch.where(most > 0.875, e - 2, e - 3)
    e = torch.where(most == 0, -127, e).clamp(-127, 125)
    # a power of two at a time: 2^-e alone may leave fp32's range
    a = torch.ldexp(torch.ldexp(x.abs(), -(e // 2)[..., None]), -(e - e // 2)[..., None])
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    code = code + 8 * (x < 0).to(torch.uint8)
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _page_bytes(page, kv_heads, dim):
    return kv_heads * page * -(-dim // GROUP) * 34


def _planes(pool, page, kv_heads, dim):
    """Views of pool bytes [pages, page_bytes] by key head: K codes, V codes [pages, kv_heads, tiles, groups, 16
    tokens, 16 bytes], K scales, V scales [pages, kv_heads, tiles, groups, 16 tokens]."""
    groups, tiles = -(-dim // GROUP), page // TILE
    head = pool.view(pool.shape[0], kv_heads, -1)
    n = page * groups
    codes = (pool.shape[0], kv_heads, tiles, groups, TILE, 16)
    return (head[..., : 16 * n].view(codes), head[..., 16 * n: 32 * n].view(codes),
            head[..., 32 * n: 33 * n].view(codes[:-1]), head[..., 33 * n:].view(codes[:-1]))


def _put(pool, page, rows, x, which):
    """Writes x [tokens, kv_heads, dim] to token places ``rows`` (int64) of pool as K (which 0) or V (1)."""
    kv_heads, dim = x.shape[1:]
    planes = _planes(pool, page, kv_heads, dim)
    code, scale = _encode(x)
    code = code.unflatten(-1, (-1, 16, 2))
    pair = code[..., 0] | code[..., 1] << 4
    at, tile, slot = rows // page, rows % page // TILE, rows % TILE
    planes[which][at, :, tile, :, slot] = pair
    planes[2 + which][at, :, tile, :, slot] = scale


def _get(pool, page, rows, kv_heads, dim, which, dtype=torch.float32):
    """The values of token places ``rows`` (int64, any shape) as K or V: [*rows.shape, kv_heads, dim]."""
    planes = _planes(pool, page, kv_heads, dim)
    at, tile, slot = rows // page, rows % page // TILE, rows % TILE
    # indices apart: rows' dimensions come first
    pair, scale = planes[which][at, :, tile, :, slot], planes[2 + which][at, :, tile, :, slot]
    code = torch.stack([pair & 15, pair >> 4], -1).flatten(-2)  # [..., kv_heads, groups, 32]
    value = torch.ldexp(_levels(dtype)[code.int()], (scale.int() - 127)[..., None])
    return value.flatten(-2)[..., :dim]


# ------------------------------------------------------------------------ inputs


def _pages_state(case, seed):
    """Tables, lengths and counts of a pool in use (host arrays): sequences of different lengths, some sharing
    the first pages of another one, pages taken in no order, part of the pool free."""
    r = np.random.default_rng(seed)
    seqs, most, page, pages = case["seqs"], case["most"], case["page"], case["pages"]
    room = most + -(-case.get("new", 0) // page) + 1
    table = np.full((seqs, room), -1, dtype=np.int32)
    length, refs = np.zeros(seqs, dtype=np.int32), np.zeros(pages, dtype=np.int32)
    order, used = r.permutation(pages), 0
    for b in range(seqs):
        if b % 8 == 5:
            continue  # waits for a prompt
        n = int(r.integers(1, most * page + 1))
        own_pages, shared = -(-n // page), 0
        if b and r.random() < 0.4 and length[b - 1]:
            shared = min(own_pages, -(-int(length[b - 1]) // page))
            if shared == own_pages:  # the last page too: the same tokens
                n = min(n, int(length[b - 1]))
                own_pages = shared = -(-n // page)
        if used + own_pages - shared > 0.6 * pages:
            continue
        table[b, :shared] = table[b - 1, :shared]
        table[b, shared:own_pages] = order[used: used + own_pages - shared]
        used += own_pages - shared
        np.add.at(refs, table[b, :own_pages], 1)
        length[b] = n
    return table, length, refs


def _step_inputs(case, seed):
    """(parent of each sequence, number of new tokens of each) on the host."""
    r = np.random.default_rng(seed + 1)
    seqs = case["seqs"]
    parent = np.arange(seqs)
    if case["new"] == 1:  # beams: groups of four take their parents among themselves
        parent = parent // 4 * 4 + r.integers(0, 4, seqs)
        parent = np.minimum(parent, seqs - 1)
    if case["ended"]:
        parent[r.permutation(seqs)[: case["ended"]]] = -1
    new = np.ones(seqs, dtype=np.int64)
    if case["new"] > 1:  # waiting sequences get their prompts
        waiting = len(new[5::8])
        new[5::8] = r.permutation(1 + np.arange(waiting) * case["new"] // max(waiting, 1))
    return parent.astype(np.int32), np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    s = {"case": case}
    if case["op"] == "int8":
        m, k, n = case["tokens"], case["k"], case["n"]
        room = -(-k // 256) * 256  # rows of int8 tokens end in zeros up to a multiple of 256

        def codes(rows):
            out, scale = torch.zeros(rows, room, dtype=torch.int8, device=DEV), []
            for part in range(0, rows, 8192):
                x = normal(min(8192, rows - part), k)
                top = x.abs().amax(1)
                out[part: part + x.shape[0], :k] = (x * (127 / top)[:, None]).round().clamp(-127, 127).to(torch.int8)
                scale.append(top / 127)
            return out, torch.cat(scale)

        x, x_scale = codes(m)
        w, w_scale = codes(n)
        s.update(x=x, x_scale=x_scale, x_sum=x.sum(1, dtype=torch.int32), w=w[:, :k].contiguous(),
                 w_scale=w_scale / math.sqrt(k), bias=normal(n) if case["bias"] else None,
                 out=torch.empty(m, n, dtype=TYPES[case["out"]], device=DEV))
        return s
    if case["op"] in ("step", "compact"):
        table, length, refs = _pages_state(case, seed)
        flat = np.concatenate([table.ravel(), length, refs, [0]])
        s.update(state0=_i32(flat), shape=table.shape,
                 pool=torch.randint(0, 256, (case["layers"], case["pages"], case["page_bytes"]), generator=g,
                                    device=DEV, dtype=torch.uint8))
        if case["op"] == "step":
            parent, q_start = _step_inputs(case, seed)
            s.update(parent=_i32(parent), q_start=_i32(q_start), tokens=int(q_start[-1]))
        return s
    kv_heads, dim, page, kind = case["kv_heads"], case["dim"], case["page"], TYPES[case["type"]]
    r = np.random.default_rng(seed)
    channel = torch.exp(0.5 * normal(2, kv_heads, dim))  # channels of different size, as keys have
    if case["op"] == "write":
        m, room = case["tokens"], case["pages"] * page
        rows = r.permutation(room)[:m]
        if m <= 64:
            rows[:: max(2, m // 3)] = -1  # padding tokens of a fixed batch
        pool = torch.zeros(case["pages"] + 1, _page_bytes(page, kv_heads, dim), dtype=torch.uint8, device=DEV)
        _put(pool, page, torch.arange(room, device=DEV), normal(room, kv_heads, dim), 0)
        _put(pool, page, torch.arange(room, device=DEV), normal(room, kv_heads, dim), 1)
        # the last page takes what the plain form writes for padding
        s.update(k=(normal(m, kv_heads, dim) * channel[0]).to(kind), v=(normal(m, kv_heads, dim) * channel[1]).to(kind),
                 rows=_i32(rows), every=_i32(np.arange(room)), pool=pool)
        return s
    q_len, k_len = _ints(case["q"]), _ints(case["k"])
    q_start = np.concatenate([[0], np.cumsum(q_len)])
    need = [-(-n // page) for n in k_len]
    pages = sum(need) + 3
    order, table, at = r.permutation(pages), np.full((len(k_len), max(need) + 1), -1, dtype=np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    pool = torch.zeros(pages, _page_bytes(page, kv_heads, dim), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (page * kv_heads * dim))
    for which in (0, 1):
        for lo in range(0, pages, step):
            rows = torch.arange(lo * page, min(pages, lo + step) * page, device=DEV)
            _put(pool, page, rows, normal(len(rows), kv_heads, dim) * channel[which], which)
    t = int(q_start[-1])
    s.update(q=normal(t, case["heads"], dim).to(kind), pool=pool, table=_i32(table), q_start=_i32(q_start),
             k_len=_i32(k_len), most_q=max(q_len), most_k=max(k_len),
             out=torch.empty(t, case["heads"], dim, dtype=TYPES[case["out"]], device=DEV),
             lse=torch.empty(t, case["heads"], device=DEV))
    return s


# ------------------------------------------------------------------ plain forms


def _plain_int8(s):
    k = s["case"]["k"]
    y = s["x"][:, :k].float() @ s["w"].float().t()
    y = y * (s["x_scale"][:, None] * s["w_scale"])
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[s["case"]["out"]])


def _plain_write(s):
    c, pool, page = s["case"], s["pool"], s["case"]["page"]
    rows = torch.where(s["rows"] < 0, c["pages"] * page, s["rows"]).long()
    _put(pool, page, rows, s["k"], 0)
    _put(pool, page, rows, s["v"], 1)
    return tuple(_get(pool, page, s["every"].long(), c["kv_heads"], c["dim"], which).bfloat16() for which in (0, 1))


def _plain_attention(s):
    c, q = s["case"], s["q"]
    t, heads, dim = q.shape
    kv, page, most_q, most_k = c["kv_heads"], c["page"], s["most_q"], s["most_k"]
    first, n_q = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    n_k = s["k_len"].long()
    iq, ik = torch.arange(most_q, device=DEV), torch.arange(most_k, device=DEV)
    qs = q.float()[(first[:, None] + iq).clamp(max=t - 1)]
    at = s["table"].long()[:, ik // page].clamp(min=0) * page + ik % page
    ks, vs = (_get(s["pool"], page, at, kv, dim, which) for which in (0, 1))
    n, group = qs.shape[0], heads // kv
    qs = qs.reshape(n, most_q, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kv, group * most_q, dim)
    score = qs @ ks.permute(0, 2, 3, 1) * dim ** -0.5
    sees = ik < n_k[:, None, None]
    if c["causal"]:
        sees = sees & (ik <= (n_k - n_q)[:, None, None] + iq[:, None])
    sees = sees.expand(n, most_q, most_k)[:, None, None]
    score = score.reshape(n, kv, group, most_q, most_k).masked_fill_(~sees, -math.inf)
    score = score.reshape(n, kv, group * most_q, most_k)
    if most_k:
        top = score.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
    else:
        top = torch.zeros(score.shape[:-1] + (1,), device=DEV)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = p @ vs.permute(0, 2, 1, 3)
    out = out / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    row = torch.arange(t, device=DEV)
    seq = (row[:, None] >= s["q_start"][1:]).sum(-1).clamp(max=n - 1)
    out = out.reshape(n, heads, most_q, dim)[seq, :, row - first[seq]]
    return out.to(TYPES[c["out"]]), lse.reshape(n, heads, most_q)[seq, :, row - first[seq]]


def _split_state(s):
    seqs, room = s["shape"]
    state = s["state0"].clone()
    n = seqs * room
    return state[:n].view(seqs, room).clone(), state[n: n + seqs].clone(), state[n + seqs: -1].clone()


def _counts(table, length, page, pages):
    used = torch.arange(table.shape[1], device=DEV) * page < length[:, None]
    counts = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
    return counts.index_add_(0, torch.where(used, table, pages).flatten(), used.flatten().int())[:pages]


def _plain_step(s):
    c = s["case"]
    table, length, _ = _split_state(s)
    page, pages, room = c["page"], c["pages"], s["shape"][1]
    # fork
    alive = (s["parent"] >= 0) & (s["parent"] < len(length))
    parent = s["parent"].clamp(0, len(length) - 1).long()
    length = torch.where(alive, length[parent], 0)
    table = torch.where(alive[:, None], table[parent], -1)
    refs = _counts(table, length, page, pages)
    # grow
    new = s["q_start"][1:] - s["q_start"][:-1]
    have, want = (length + page - 1) // page, (length + new + page - 1) // page
    seq = torch.arange(len(length), device=DEV)
    last = (have - 1).clamp(min=0).long()
    tail = table[seq, last].clamp(min=0)
    part = (new > 0) & (length % page != 0) & (refs[tail.long()] > 1)
    need = want - have + part.int()
    fits = want <= room
    need = torch.where(fits, need, 0)
    free = (refs == 0).nonzero()[:, 0].int()
    ends = need.cumsum(0)
    granted = fits & ((need == 0) | (ends <= len(free)))
    part = part & granted
    start = ends - need
    slots = torch.arange(room, device=DEV)
    begin = (have - part.int())[:, None]
    fresh = granted[:, None] & (slots >= begin) & (slots < want[:, None])
    pick = (start[:, None] + slots - begin).clamp(0, max(len(free) - 1, 0)).long()
    copied = part.nonzero()[:, 0]
    source = tail[copied].long()
    if len(free):
        table = torch.where(fresh, free[pick], table)
    target = table[copied, last[copied]].long()
    s["pool"][:, target] = s["pool"][:, source]
    granted_new = torch.where(granted, new, 0)
    length = length + granted_new
    refs = _counts(table, length, page, pages)
    token = torch.arange(s["tokens"], device=DEV)
    seq = (token[:, None] >= s["q_start"][1:]).sum(-1)
    position = length[seq] - granted_new[seq] + token - s["q_start"][seq]
    row = table[seq, (position // page).clamp(0, room - 1).long()] * page + position % page
    row = torch.where(granted[seq], row, -1)
    return (table, length.int(), refs, row.int(), position.int(), granted_new.int(), s["pool"])


def _plain_compact(s):
    c = s["case"]
    table, length, refs = _split_state(s)
    live = refs > 0
    n = int(live.sum())
    index = torch.arange(c["pages"], device=DEV)
    source, target = (live & (index >= n)).nonzero()[:, 0], (~live & (index < n)).nonzero()[:, 0]
    s["pool"][:, target] = s["pool"][:, source]
    moved = index.clone()
    moved[source] = target
    table = torch.where(table >= 0, moved[table.clamp(min=0).long()].int(), table)
    refs[target] = refs[source]
    refs[source] = 0
    return table, length, refs, s["pool"]


# ---------------------------------------------------------------- the operators


def _own_int8(s):
    import bit_ternary_weight_absmean_amd as bt

    if "weight" not in s:  # laid out once, as a program that loads a model does
        s["weight"] = bt.pack_int8(s["w"], s["w_scale"])
        s["workspace"] = bt.int8_workspace(s["x"].shape[0], s["weight"])
    return bt.int8_gemm(s["weight"], (s["x"], s["x_scale"], s["x_sum"]), bias=s["bias"], out=s["out"],
                        workspace=s["workspace"])


def _own_write(s):
    import bit_ternary_weight_absmean_amd as bt

    c = s["case"]
    if "cache" not in s:
        s["cache"] = bt.Cache4(c["pages"], c["page"], c["kv_heads"], c["dim"], data=s["pool"][None, :-1])
        room = c["pages"] * c["page"]
        s["read"] = tuple(torch.empty(room, c["kv_heads"], c["dim"], dtype=torch.bfloat16, device=DEV)
                          for _ in range(2))
    bt.cache4_write(s["cache"], s["k"], s["v"], s["rows"])
    return bt.cache4_read(s["cache"], s["every"], out=s["read"])


def _own_attention(s):
    import bit_ternary_weight_absmean_amd as bt

    c = s["case"]
    if "cache" not in s:
        s["cache"] = bt.Cache4(s["pool"].shape[0], c["page"], c["kv_heads"], c["dim"], data=s["pool"][None])
        s["workspace"] = bt.attention4_workspace(s["q"], s["cache"], s["table"])
    return bt.attention4(s["q"], s["cache"], s["table"], s["k_len"], s["q_start"], causal=c["causal"], out=s["out"],
                         lse=s["lse"], workspace=s["workspace"])


def _own_pages(s):
    import bit_ternary_weight_absmean_amd as bt

    c = s["case"]
    if "pages" not in s:
        seqs, room = s["shape"]
        s["pages"] = bt.Pages(seqs, room, c["pages"], c["page"], device=DEV)
        if c["op"] == "step":
            s["grown"] = tuple(torch.empty(n, dtype=torch.int32, device=DEV) for n in (s["tokens"], s["tokens"], seqs))
    pages = s["pages"]
    pages.state.copy_(s["state0"])
    if c["op"] == "compact":
        bt.pages_compact(pages, s["pool"])
        return pages.table, pages.length, pages.refs, s["pool"]
    bt.pages_fork(pages, s["parent"])
    row, position, granted = bt.pages_grow(pages, s["q_start"], s["pool"], out=s["grown"])
    return pages.table, pages.length, pages.refs, row, position, granted, s["pool"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"int8": _own_int8, "write": _own_write, "attention": _own_attention, "step": _own_pages,
                "compact": _own_pages}[op](state)
    return {"int8": _plain_int8, "write": _plain_write, "attention": _plain_attention, "step": _plain_step,
            "compact": _plain_compact}[op](state)


def _copies(case, seed=1):
    """Pages that the case copies (for a usual seed: their number hardly changes)."""
    table, length, refs = _pages_state(case, seed)
    if case["op"] == "compact":
        n = int((refs > 0).sum())
        return int((refs[n:] > 0).sum())
    return len(_step_exact(case, seed)[6])


def work(case):
    if case["op"] == "int8":
        m, k, n = case["tokens"], case["k"], case["n"]
        return {"bytes": m * k + n * k + 4 * (m + n) + (4 * n if case["bias"] else 0) + SIZE[case["out"]] * m * n,
                "flops": 2.0 * m * n * k}
    if case["op"] in ("step", "compact"):
        table, _, refs = _pages_state(case, 1)
        return {"bytes": 8 * table.size + 8 * refs.size + 2 * _copies(case) * case["layers"] * case["page_bytes"],
                "flops": float(table.size)}
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    token = _page_bytes(page, kv, dim) // page
    if case["op"] == "write":
        values = 2 * kv * dim
        return {"bytes": case["tokens"] * (values * SIZE[case["type"]] + token) + case["pages"] * page *
                (token + 2 * values), "flops": 8.0 * values * case["tokens"]}
    q_len, k_len, heads = _ints(case["q"]), _ints(case["k"]), case["heads"]
    t, pairs = sum(q_len), 0
    for n_q, n_k in zip(q_len, k_len):
        if case["causal"]:
            rows = min(n_q, n_k)
            pairs += rows * (n_k - rows + 1) + rows * (rows - 1) // 2
        else:
            pairs += n_q * n_k
    return {"bytes": t * heads * dim * (SIZE[case["type"]] + SIZE[case["out"]]) + token * sum(k_len) + 4 * t * heads,
            "flops": 4.0 * dim * heads * pairs}


# ------------------------------------------------- the definitions, in 64 bits


def _nearest(x):
    """The 4-bit value of each of x [..., 32 values of a group] (fp64), by looking at every candidate."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(top, -127.0)
    for _ in range(2):  # log2 to find the exponent, then put right what its rounding missed
        e = torch.maximum(e, torch.ceil(torch.log2(top / 7)) - 1)
        e = torch.where(top > 7 * torch.exp2(e), e + 1, e)
    e = torch.where(top == 0, -127.0, e).clamp(-127, 125)
    level = _levels(torch.float64)[:8]
    # the nearest level; of two equally near ones that with the even number
    gap = (x.abs()[..., None] * torch.exp2(-e)[..., None] - level).abs()
    gap = torch.cat([gap[..., 0::2], gap[..., 1::2]], -1)
    best = torch.cat([level[0::2], level[1::2]])[gap.argmin(-1)]
    return torch.where(x < 0, -best, best) * torch.exp2(e)


def _write_exact(case, seed):
    s = prepare(case, seed)
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    kept = (s["rows"] >= 0).nonzero()[:, 0]
    place = s["rows"][kept].long()
    out = []
    for which, x in enumerate((s["k"], s["v"])):
        old = _unpack(s["pool"], page, kv, dim, which)[: case["pages"] * page]
        if len(kept):
            value = torch.nn.functional.pad(x[kept].double(), (0, -dim % GROUP))
            for part in range(0, len(kept), 2048):
                rows = value[part: part + 2048]
                old[place[part: part + 2048]] = torch.cat([_nearest(g) for g in rows.split(GROUP, -1)], -1)[..., :dim]
        out.append(old)
    return tuple(out)


def _unpack(pool, page, kv, dim, which):
    """All tokens' values [pages * page, kv, dim] (fp64), from the byte positions of the format."""
    groups = -(-dim // GROUP)
    token, head, d = (torch.arange(n, device=DEV) for n in (page, kv, dim))
    token, head, d = token[:, None, None], head[None, :, None], d[None, None, :]
    chunk = (token // TILE * groups + d // GROUP) * TILE + token % TILE
    base = head * (page * groups * 34)
    byte = base + which * page * groups * 16 + chunk * 16 + d % GROUP // 2
    scale = base + (32 + which) * page * groups + chunk
    code = (pool[:, byte] >> (4 * (d % 2)).to(torch.uint8)) & 15
    return (_levels(torch.float64)[code.long()] * torch.exp2(pool[:, scale].double() - 127)).flatten(0, 1)


def _step_exact(case, seed):
    """The step by its rules, one sequence and page at a time (host)."""
    table, length, _ = _pages_state(case, seed)
    parent, q_start = _step_inputs(case, seed)
    page, pages, seqs = case["page"], case["pages"], case["seqs"]
    room = table.shape[1]
    held = [[int(v) for v in table[b, : -(-int(length[b]) // page)]] for b in range(seqs)]
    length = [int(v) for v in length]
    held = [list(held[p]) if 0 <= p < seqs else [] for p in parent]
    length = [length[p] if 0 <= p < seqs else 0 for p in parent]
    refs = [0] * pages
    for pages_of in held:
        for p in pages_of:
            refs[p] += 1
    free = [p for p in range(pages) if refs[p] == 0]
    asked, granted, copies, before = 0, [], [], list(refs)
    for b in range(seqs):
        n = int(q_start[b + 1] - q_start[b])
        want = -(-(length[b] + n) // page)
        copy = bool(n and length[b] % page and before[held[b][-1]] > 1)
        need = want - len(held[b]) + copy
        if want > room:
            granted.append(0)
            continue
        asked += need
        if need and asked > len(free):
            granted.append(0)
            continue
        take = free[asked - need: asked]
        if copy:
            copies.append((held[b][-1], take[0]))
            refs[held[b][-1]] -= 1
            held[b][-1] = take[0]
            held[b] += take[1:]
        else:
            held[b] += take
        for p in take:
            refs[p] += 1
        length[b] += n
        granted.append(n)
    out = np.full((seqs, room), -1, dtype=np.int32)
    rows, positions = [], []
    for b in range(seqs):
        out[b, : len(held[b])] = held[b]
        for i in range(int(q_start[b + 1] - q_start[b])):
            at = length[b] - granted[b] + i
            positions.append(at)
            rows.append(held[b][at // page] * page + at % page if granted[b] else -1)
    return out, length, refs, rows, positions, granted, copies


def exact(case, seed):
    if case["op"] == "write":
        return _write_exact(case, seed)
    s = prepare(case, seed)
    if case["op"] == "int8":
        y = torch.empty(case["tokens"], case["n"], dtype=torch.float64, device=DEV)
        x = s["x"].double()[:, : case["k"]]
        for lo in range(0, case["n"], 8192):
            part = slice(lo, min(case["n"], lo + 8192))
            y[:, part] = x @ s["w"][part].double().T * s["x_scale"].double()[:, None] * s["w_scale"][part].double()
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "step":
        *numbers, copies = _step_exact(case, seed)
        pool = s["pool"].clone()
        for src, dst in copies:
            pool[:, dst] = s["pool"][:, src]
        return tuple(_i32(v) for v in numbers) + (pool,)
    if case["op"] == "compact":
        table, length, refs = _pages_state(case, seed)
        n = int((refs > 0).sum())
        holes = [p for p in range(n) if refs[p] == 0]
        goes = dict(zip([p for p in range(n, case["pages"]) if refs[p]], holes))
        for src, dst in goes.items():
            refs[dst], refs[src] = refs[src], 0
            s["pool"][:, dst] = s["pool"][:, src]
        table = [[goes.get(int(p), int(p)) for p in row] for row in table]
        return _i32(table), _i32(length), _i32(refs), s["pool"]
    heads, kv, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n_q, n_k) in enumerate(zip(_ints(case["q"]), _ints(case["k"]))):
        used = s["table"][b, : -(-n_k // page)].long()
        ks, vs = (_unpack(s["pool"][used], page, kv, dim, which)[:n_k] for which in (0, 1))
        future = torch.ones(n_q, n_k, dtype=torch.bool, device=DEV).triu(n_k - n_q + 1)
        for j in range(heads if n_k else 0):
            h = j // (heads // kv)
            logit = s["q"][at: at + n_q, j].double() @ ks[:, h].T / math.sqrt(dim)
            if case["causal"]:
                logit[future] = -math.inf
            lse[at: at + n_q, j] = torch.logsumexp(logit, -1)
            out[at: at + n_q, j] = torch.nan_to_num(torch.softmax(logit, -1), nan=0.0) @ vs[:, h]
        at += n_q
    return out, lse
