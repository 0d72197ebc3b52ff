"""Measured cases of the attention-block operators: low-rank adapters beside a projection,
per-head norms with the position rotation, attention over packed prompts and cached keys, and
attention of a batch that shares a prefix.

``run`` computes a case in plain torch operations, or, with ``own`` set, through this
package's operators. Sizes are the package's 2B / 7B / 100B class layers (hidden 2560 / 4096 /
8192 with 20/5, 32/32 and 64/8 heads of 128) and generic ones around them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # One decode step's fused QKV projection of a 2B class model, one request.
        {"name": "adapters 1 token 2B qkv", "op": "lora", "tokens": 1, "k": 2560, "groups": "2560,640,640",
         "rank": 16, "adapters": 4, "type": "bf16", "order": "mixed", "ragged": False},
        # A decode batch of 64 requests with adapters of their own at the 7B down projection; some have none.
        {"name": "adapters 64 requests 7B down", "op": "lora", "tokens": 64, "k": 11008, "groups": "4096",
         "rank": 64, "adapters": 48, "type": "fp16", "order": "mixed", "ragged": True},
        # Packed prompts of eight tenants at the 2B gate+up projection.
        {"name": "adapters prompts 2B gate_up", "op": "lora", "tokens": 2048, "k": 2560, "groups": "6912,6912",
         "rank": 32, "adapters": 8, "type": "bf16", "order": "runs", "ragged": False},
        # One decode step of one request, 2B class.
        {"name": "norm+rope 1 token 2B", "op": "qk", "tokens": 1, "heads": 20, "kv_heads": 5, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "type": "bf16", "max_pos": 4096, "cache": 0},
        # A decode batch written into its cache rows, half-rotated heads, far positions, padding tokens.
        {"name": "norm+rope 37 tokens to cache", "op": "qk", "tokens": 37, "heads": 32, "kv_heads": 32, "dim": 128,
         "rot": 64, "interleaved": True, "norm": True, "type": "fp16", "max_pos": 1000000, "cache": 1500},
        # A large prefill batch of a 100B class model.
        {"name": "norm+rope 16384 tokens 100B", "op": "qk", "tokens": 16384, "heads": 64, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "norm": True, "type": "bf16", "max_pos": 32768, "cache": 0},
        # One request's next token, 2B class: latency.
        {"name": "attention 1 token, 777 keys", "op": "attention", "q": "1", "k": "777", "slab": 1024, "heads": 20,
         "kv_heads": 5, "dim": 128, "type": "bf16", "causal": True, "prefix": 0},
        # A decode batch over cache slabs filled to different lengths, one of them empty.
        {"name": "attention decode 64 x 8192", "op": "attention", "q": ",".join(["1"] * 64),
         "k": ",".join(str((i * 2654435761 + 97) % 8192 if i != 13 else 0) for i in range(63)) + ",8192",
         "slab": 8192, "heads": 20, "kv_heads": 5, "dim": 128, "type": "bf16", "causal": True, "prefix": 0},
        # A prefill batch of 2048 tokens in packed prompts.
        {"name": "attention packed prompts 2B", "op": "attention", "q": "611,1,300,1024,112", "k": "611,1,300,1024,112",
         "slab": 0, "heads": 20, "kv_heads": 5, "dim": 128, "type": "bf16", "causal": True, "prefix": 0},
        # One long prompt, 7B class.
        {"name": "attention prompt 8192 7B", "op": "attention", "q": "8192", "k": "8192", "slab": 0, "heads": 32,
         "kv_heads": 32, "dim": 128, "type": "fp16", "causal": True, "prefix": 0},
        # A few requests behind one system prompt.
        {"name": "prefix 1000, 8 requests", "op": "attention", "q": ",".join(["1"] * 8), "k": "1,200,0,33,64,7,129,90",
         "slab": 200, "heads": 32, "kv_heads": 32, "dim": 128, "type": "fp16", "causal": True, "prefix": 1000},
        # A decode batch behind one long document, 100B class.
        {"name": "prefix 16384, 64 requests", "op": "attention", "q": ",".join(["1"] * 64),
         "k": ",".join(str((i * 331 + 5) % 512 + 1) for i in range(64)), "slab": 512, "heads": 64, "kv_heads": 8,
         "dim": 128, "type": "bf16", "causal": True, "prefix": 16384},
    ]


HEADS = [(20, 5, 128), (32, 32, 128), (64, 8, 128), (16, 2, 64), (8, 1, 256), (6, 3, 80), (12, 4, 96)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "qk", "attention", "attention", "prefix"])
    if op == "lora":
        tokens = _log(rng, 1, 2048)
        groups = [_log(rng, 64, 6912) for _ in range(rng.choice([1, 1, 2, 3]))]
        rank = rng.choice([1, 4, 8, 8, 12, 16, 16, 32, 64])
        return {"op": "lora", "tokens": tokens, "k": _log(rng, 64, 11008), "groups": ",".join(map(str, groups)),
                "rank": rank, "adapters": _log(rng, 1, 64), "type": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "order": rng.choice(["mixed", "runs"]), "ragged": rng.random() < 0.3}
    heads, kv_heads, dim = rng.choice(HEADS)
    if op == "qk":
        tokens = _log(rng, 1, 12000)
        return {"op": "qk", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim, 8 * max(1, dim // 16)]), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.75, "type": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "max_pos": _log(rng, 16, 2000000), "cache": rng.choice([0, 0, 3 * tokens + 11])}
    kind = rng.choice(["bf16", "fp16"])
    if op == "prefix":
        n = _log(rng, 1, 64)
        q = [rng.choice([1, 1, 1, 2, 4]) for _ in range(n)]
        slab = _log(rng, 8, 600)
        return {"op": "attention", "q": ",".join(map(str, q)),
                "k": ",".join(str(rng.randint(0, slab)) for _ in q), "slab": slab, "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "type": kind, "causal": True, "prefix": _log(rng, 16, 12000)}
    if rng.random() < 0.5:  # decode, drafts of a few tokens, a continued prompt
        n = _log(rng, 1, 96)
        slab = _log(rng, 16, 6000)
        most = rng.choice([1, 1, 4, 33])
        q = [rng.randint(min(1, most - 1), most) for _ in range(n)]
        q[rng.randrange(n)] = most
        return {"op": "attention", "q": ",".join(map(str, q)), "k": ",".join(str(rng.randint(0, slab)) for _ in q),
                "slab": slab, "heads": heads, "kv_heads": kv_heads, "dim": dim, "type": kind, "causal": True,
                "prefix": 0}
    q = [_log(rng, 1, 2200) for _ in range(rng.randint(1, 5))]
    return {"op": "attention", "q": ",".join(map(str, q)), "k": ",".join(map(str, q)), "slab": 0, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "type": kind, "causal": rng.random() < 0.85, "prefix": 0}


def _ints(text):
    return [int(v) for v in text.split(",")]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _lora_sets(case, seed):
    """(adapter of each token, rank of each adapter) on the host."""
    r = np.random.default_rng(seed)
    m, n = case["tokens"], case["adapters"]
    index = r.integers(0, n, m)
    if case["order"] == "runs":  # tokens of one prompt are neighbours
        index = (np.arange(m) * n // max(m, 1) + int(r.integers(0, n))) % n
    elif m > 8:
        index[r.random(m) < 0.06] = -1  # requests without an adapter
    ranks = r.integers(1, case["rank"] + 1, n) if case["ragged"] else np.full(n, case["rank"])
    return index.astype(np.int32), ranks.astype(np.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    s = {"case": case, "type": TYPES[case["type"]]}
    if case["op"] == "lora":
        m, k, rank, n_ad, groups = case["tokens"], case["k"], case["rank"], case["adapters"], _ints(case["groups"])
        n = sum(groups)
        index, ranks = _lora_sets(case, seed)
        s.update(groups=groups, x=normal(m, k), base=normal(m, n), index=_i32(index),
                 ranks=_i32(ranks) if case["ragged"] else None,
                 a=(normal(n_ad, len(groups) * rank, k) / math.sqrt(k)).to(s["type"]),
                 b=(normal(n_ad, n, rank) / math.sqrt(rank)).to(s["type"]),
                 scale=torch.rand(n_ad, generator=g, device=DEV) + 0.5, out=torch.empty(m, n, device=DEV))
        return s
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        m, cap = case["tokens"], case["cache"]
        half = case["rot"] // 2
        pos = torch.randint(0, case["max_pos"], (m,), generator=g, device=DEV, dtype=torch.int32)
        s.update(qkv=normal(m, (heads + 2 * kv_heads) * dim), positions=pos,
                 inv_freq=10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half),
                 q_weight=1 + 0.1 * normal(dim) if case["norm"] else None,
                 k_weight=1 + 0.1 * normal(dim) if case["norm"] else None, rows=None,
                 q=torch.empty(m, heads, dim, dtype=s["type"], device=DEV))
        room = cap + 1 if cap else m  # the last row of a cache takes what the plain form writes for padding
        s.update(k=normal(room, kv_heads, dim).to(s["type"]), v=normal(room, kv_heads, dim).to(s["type"]))
        if cap:
            rows = np.random.default_rng(seed).permutation(cap)[:m]
            if m > 4:
                rows[:: max(2, m // 3)] = -1  # padding tokens of a fixed batch
            s.update(rows=_i32(rows), k_room=s["k"], v_room=s["v"], k=s["k"][:cap], v=s["v"][:cap])
        return s
    q_len, k_len = _ints(case["q"]), _ints(case["k"])
    slab = case["slab"]
    q_start = np.concatenate([[0], np.cumsum(q_len)])
    k_start = np.arange(len(k_len)) * slab if slab else np.concatenate([[0], np.cumsum(k_len)[:-1]])
    t, room = int(q_start[-1]), len(k_len) * slab if slab else sum(k_len)
    kind = s["type"]
    s.update(q=normal(t, heads, dim).to(kind), k=normal(room, kv_heads, dim).to(kind),
             v=normal(room, kv_heads, dim).to(kind), q_start=_i32(q_start), k_start=_i32(k_start), k_len=_i32(k_len),
             most_q=max(q_len), most_k=max(k_len), out=torch.empty(t, heads, dim, dtype=kind, device=DEV),
             lse=torch.empty(t, heads, device=DEV), prefix_k=None, prefix_v=None)
    if case["prefix"]:
        s.update(prefix_k=normal(case["prefix"], kv_heads, dim).to(kind),
                 prefix_v=normal(case["prefix"], kv_heads, dim).to(kind))
    return s


# ------------------------------------------------------------------ plain forms


def _plain_lora(s):
    x, a, b, groups = s["x"], s["a"].float(), s["b"].float(), s["groups"]
    n_ad, rank = b.shape[0], b.shape[2]
    n, n_gr = b.shape[1], len(groups)
    h = (x @ a.reshape(-1, a.shape[2]).t()).reshape(-1, n_ad, n_gr, rank)
    mine = s["index"].long()[:, None] == torch.arange(n_ad, device=DEV)
    keep = (mine * s["scale"])[:, :, None, None]
    if s["ranks"] is not None:
        keep = keep * (torch.arange(rank, device=DEV) < s["ranks"][:, None])[None, :, None, :]
    group = torch.repeat_interleave(torch.arange(n_gr, device=DEV), torch.tensor(groups, device=DEV), output_size=n)
    one = (group[:, None] == torch.arange(n_gr, device=DEV)).float()
    wide = b.permute(1, 0, 2)[:, :, None, :] * one[:, None, :, None]
    return s["base"] + (h * keep).reshape(h.shape[0], -1) @ wide.reshape(n, -1).t()


def _plain_rotate(x, cos, sin, rot, interleaved):
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., : rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([part, rest], -1)


def _plain_qk(s):
    c = s["case"]
    hq, hk, dim = c["heads"], c["kv_heads"], c["dim"]
    x = s["qkv"].float().reshape(-1, hq + 2 * hk, dim)
    q, k, v = x[:, :hq], x[:, hq: hq + hk], x[:, hq + hk:]
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["q_weight"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["k_weight"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _plain_rotate(q, cos, sin, c["rot"], c["interleaved"]).to(s["type"])
    k = _plain_rotate(k, cos, sin, c["rot"], c["interleaved"]).to(s["type"])
    v = v.to(s["type"])
    if s["rows"] is None:
        return q, k, v
    room = c["cache"]
    at = torch.where(s["rows"] < 0, room, s["rows"]).long()
    s["k_room"][at] = k
    s["v_room"][at] = v
    return q, s["k"], s["v"]


def _plain_attention(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    t, heads, dim = q.shape
    kv = k.shape[1]
    most_q, most_k = s["most_q"], s["most_k"]
    first, n_q = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    n_k = s["k_len"].long()
    iq, ik = torch.arange(most_q, device=DEV), torch.arange(most_k, device=DEV)
    qs = q.float()[(first[:, None] + iq).clamp(max=t - 1)]
    at = (s["k_start"].long()[:, None] + ik.clamp(max=max(most_k - 1, 0))).clamp(max=max(k.shape[0] - 1, 0))
    ks, vs = k[at].float(), v[at].float()
    n, group = qs.shape[0], heads // kv
    qs = qs.reshape(n, most_q, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kv, group * most_q, dim)
    score = qs @ ks.permute(0, 2, 3, 1) * dim ** -0.5
    sees = ik < n_k[:, None, None]
    if c["causal"]:
        sees = sees & (ik <= (n_k - n_q)[:, None, None] + iq[:, None])
    sees = sees.expand(n, most_q, most_k)[:, None, None]
    score = score.reshape(n, kv, group, most_q, most_k).masked_fill_(~sees, -math.inf)
    score = score.reshape(n, kv, group * most_q, most_k)
    if s["prefix_k"] is not None:
        score = torch.cat([qs @ s["prefix_k"].float().permute(1, 2, 0) * dim ** -0.5, score], -1)
    if score.shape[-1]:
        top = score.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
    else:
        top = torch.zeros(score.shape[:-1] + (1,), device=DEV)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    far = c["prefix"]
    out = p[..., far:] @ vs.permute(0, 2, 1, 3)
    if far:
        out = out + p[..., :far] @ s["prefix_v"].float().permute(1, 0, 2)
    out = out / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    row = torch.arange(t, device=DEV)
    seq = (row[:, None] >= s["q_start"][1:]).sum(-1).clamp(max=n - 1)
    out = out.reshape(n, heads, most_q, dim)[seq, :, row - first[seq]]
    return out.to(s["type"]), lse.reshape(n, heads, most_q)[seq, :, row - first[seq]]


# ---------------------------------------------------------------- the operators


def _own_lora(s):
    import bit_ternary_weight_absmean_amd as bt

    if "adapters" not in s:  # made once, as a program that serves them does
        s["adapters"] = bt.LoraAdapters(s["a"], s["b"], s["scale"], ranks=s["ranks"], group_rows=s["groups"])
        s["workspace"] = bt.lora_workspace(s["x"].shape[0], s["adapters"])
    return bt.lora_apply(s["x"], s["adapters"], s["index"], base=s["base"], out=s["out"], workspace=s["workspace"])


def _own_qk(s):
    import bit_ternary_weight_absmean_amd as bt

    c = s["case"]
    return bt.qk_norm_rope(s["qkv"], s["positions"], s["inv_freq"], c["heads"], c["kv_heads"],
                           q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6, interleaved=c["interleaved"],
                           rows=s["rows"], out=(s["q"], s["k"], s["v"]))


def _own_attention(s):
    import bit_ternary_weight_absmean_amd as bt

    if "workspace" not in s:
        s["workspace"] = bt.attention_workspace(s["q"], s["k"], s["k_len"].shape[0], prefix_k=s["prefix_k"])
    return bt.attention(s["q"], s["k"], s["v"], s["q_start"], s["k_start"], s["k_len"], causal=s["case"]["causal"],
                        prefix_k=s["prefix_k"], prefix_v=s["prefix_v"], out=s["out"], lse=s["lse"],
                        workspace=s["workspace"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"lora": _own_lora, "qk": _own_qk, "attention": _own_attention}[op](state)
    return {"lora": _plain_lora, "qk": _plain_qk, "attention": _plain_attention}[op](state)


def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "lora":
        m, k, rank, groups = case["tokens"], case["k"], case["rank"], _ints(case["groups"])
        n, wide = sum(groups), rank * len(groups)
        used = min(case["adapters"], m)
        return {"bytes": 4 * m * k + 8 * m * n + used * size * (wide * k + n * rank),
                "flops": 2.0 * m * (wide * k + n * rank)}
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        values = case["tokens"] * (heads + 2 * kv) * dim
        return {"bytes": values * (4 + size) + 4 * case["tokens"], "flops": 8.0 * values}
    q_len, k_len, far = _ints(case["q"]), _ints(case["k"]), case["prefix"]
    t = sum(q_len)
    pairs = far * t
    for n_q, n_k in zip(q_len, k_len):
        if case["causal"]:
            seen = max(0, n_k - n_q + 1), n_k  # keys of the first and of the last query
            rows = min(n_q, n_k)
            pairs += rows * (seen[0] if n_k >= n_q else 1) + rows * (rows - 1) // 2
        else:
            pairs += n_q * n_k
    return {"bytes": size * dim * (2 * t * heads + 2 * kv * (sum(k_len) + far)) + 4 * t * heads,
            "flops": 4.0 * dim * heads * pairs}


# ------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        index, ranks = _lora_sets(case, seed)
        out = s["base"].double()
        for ad in sorted(set(index.tolist()) - {-1}):
            tok = torch.tensor(np.nonzero(index == ad)[0], device=DEV)
            r, col = int(ranks[ad]), 0
            for g, width in enumerate(s["groups"]):
                down = s["a"][ad, g * case["rank"]: g * case["rank"] + r].double()
                up = s["b"][ad, col: col + width, :r].double()
                out[tok, col: col + width] += s["scale"][ad].double() * (s["x"][tok].double() @ down.T @ up.T)
                col += width
        return out
    if case["op"] == "qk":
        hq, hk, dim, rot = case["heads"], case["kv_heads"], case["dim"], case["rot"]
        x = s["qkv"].double().view(-1, hq + 2 * hk, dim)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None, None] * s["inv_freq"])

        def head(part, weight):
            if weight is not None:
                part = part / (part.pow(2).sum(-1, keepdim=True) / dim + 1e-6).sqrt() * weight.double()
            part = part.clone()
            lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(part[..., lo].contiguous(), part[..., hi].contiguous()) * turn
            part[..., lo], part[..., hi] = z.real, z.imag
            return part

        q, k, v = head(x[:, :hq], s["q_weight"]), head(x[:, hq:hq + hk], s["k_weight"]), x[:, hq + hk:]
        if s["rows"] is None:
            return q, k, v
        kept = (s["rows"] >= 0).nonzero()[:, 0]
        k_all, v_all = s["k"].double(), s["v"].double()
        k_all[s["rows"][kept].long()], v_all[s["rows"][kept].long()] = k[kept], v[kept]
        return q, k_all, v_all
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    at, starts = 0, s["k_start"].tolist()
    for n_q, n_k, lo in zip(_ints(case["q"]), _ints(case["k"]), starts):
        future = torch.ones(n_q, n_k, dtype=torch.bool, device=DEV).triu(n_k - n_q + 1)
        for h in range(kv):
            ks, vs = s["k"][lo: lo + n_k, h].double(), s["v"][lo: lo + n_k, h].double()
            if case["prefix"]:
                ks = torch.cat([s["prefix_k"][:, h].double(), ks])
                vs = torch.cat([s["prefix_v"][:, h].double(), vs])
            for j in range(h * heads // kv, (h + 1) * heads // kv):
                logit = s["q"][at: at + n_q, j].double() @ ks.T / math.sqrt(dim)
                if case["causal"]:
                    logit[:, case["prefix"]:][future] = -math.inf
                if logit.numel():
                    lse[at: at + n_q, j] = torch.logsumexp(logit, -1)
                    out[at: at + n_q, j] = torch.nan_to_num(torch.softmax(logit, -1), nan=0.0) @ vs
        at += n_q
    return out, lse
