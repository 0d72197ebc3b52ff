"""The 4-bit cache, its pages and the int8 product by their definitions (torch in 64 bits, plain Python), for the
tests."""
import math

import torch

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def encode(x):
    """(codes 0..15, scale bytes) of x [..., D] (any float type, converted exactly): groups of 32, the last one filled
    up with zeros. All steps are exact in fp64."""
    x = torch.nn.functional.pad(x.double(), (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    odd = ~torch.isfinite(x).all(-1)
    m, e = torch.frexp(torch.where(odd, torch.ones_like(top), top))  # m in [0.5, 1): top <= 7 * 2^(e - 3) for m <= 7/8
    e = torch.where(m > 0.875, e - 2, e - 3)
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 125)
    a = x.abs() * torch.exp2(-e.double())[..., None]
    code = torch.zeros_like(a, dtype=torch.int64)
    for i in range(7):  # past the middle, or on it from an odd code
        middle = (LEVELS[i] + LEVELS[i + 1]) / 2
        code += ((a >= middle) if i % 2 else (a > middle)).long()
    code = torch.where(x.double().signbit(), code + 8, code)
    code = torch.where(odd[..., None], torch.zeros_like(code), code)
    return code.flatten(-2), torch.where(odd, torch.full_like(e, 255), e + 127).long()


def decode(code, scale, D):
    """Values (fp64) of codes [..., 32 G] and scale bytes [..., G]."""
    levels = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=code.device)
    v = levels[code.long()].unflatten(-1, (-1, 32)) * torch.exp2(scale.double() - 127)[..., None]
    v = torch.where((scale > 252)[..., None], torch.full_like(v, math.nan), v)
    return v.flatten(-2)[..., :D]


def places(row, page_tokens, kv, D):
    """Byte offsets of place `row` in its layer: ((K codes, V codes) [kv, G], (K scales, V scales) [kv, G])."""
    G = -(-D // 32)
    page, t = row // page_tokens, row % page_tokens
    head = page * kv * page_tokens * G * 34 + torch.arange(kv)[:, None] * page_tokens * G * 34
    chunk = ((t // 16) * G + torch.arange(G)[None]) * 16 + t % 16
    n = page_tokens * G
    return (head + 16 * chunk, head + 16 * n + 16 * chunk), (head + 32 * n + chunk, head + 33 * n + chunk)


def put(data, row, page_tokens, k, v):
    """Writes k, v [kv, D] of one token into a layer's bytes `data` (1-D uint8, CPU)."""
    kv, D = k.shape
    codes, scales = places(row, page_tokens, kv, D)
    for x, at, sat in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        c, s = encode(x)
        pair = (c[:, 0::2] | c[:, 1::2] << 4).to(torch.uint8).reshape(kv, -1, 16)
        data[(at[..., None] + torch.arange(16)).flatten()] = pair.flatten()
        data[sat.flatten()] = s.to(torch.uint8).flatten()


def get(data, page_tokens, kv, D):
    """All places' K and V [places, kv, D] (fp64) of a layer's bytes [pages, page_bytes] (any device)."""
    G, n = -(-D // 32), page_tokens
    pages = data.shape[0]
    head = data.reshape(pages, kv, -1)
    out = []
    for which in (0, 1):
        code = head[..., 16 * n * G * which: 16 * n * G * (which + 1)].reshape(pages, kv, n // 16, G, 16, 16)
        scale = head[..., n * G * (32 + which): n * G * (33 + which)].reshape(pages, kv, n // 16, G, 16)
        code = torch.stack([code & 15, code >> 4], -1).flatten(-2)
        # [pages, tile, token, kv, G]
        code = code.permute(0, 2, 4, 1, 3, 5).reshape(pages * n, kv, G * 32)
        scale = scale.permute(0, 2, 4, 1, 3).reshape(pages * n, kv, G)
        out.append(decode(code, scale, D))
    return out


def gather(data, table, k_len, page_tokens, kv, D):
    """(k, v, k_start) of the sequences' keys, packed (fp64), for block_ref.attention; table a list of lists. The keys
    of entries outside the cache are left out: the third value counts what is left."""
    k_all, v_all = get(data, page_tokens, kv, D)
    rows, start, left = [], [], []
    for b, n in enumerate(k_len):
        start.append(len(rows))
        for j in range(n):
            page = table[b][j // page_tokens]
            if 0 <= page < data.shape[0]:
                rows.append(page * page_tokens + j % page_tokens)
        left.append(len(rows) - start[-1])
    at = torch.tensor(rows, dtype=torch.long, device=data.device)
    return k_all[at], v_all[at], start, left


class Model:
    """The pages' bookkeeping, one sequence and page at a time. pool [layers, pages, ...] on the CPU."""

    def __init__(self, seqs, max_pages, pages, page_tokens, pool):
        self.W, self.P, self.page, self.pool = max_pages, pages, page_tokens, pool
        self.held = [[] for _ in range(seqs)]
        self.length = [0] * seqs

    def refs(self):
        refs = [0] * self.P
        for held in self.held:
            for p in held:
                refs[p] += 1
        return refs

    def table(self):
        return [h + [-1] * (self.W - len(h)) for h in self.held]

    def fork(self, parent):
        seqs = len(self.held)
        self.held = [list(self.held[p]) if 0 <= p < seqs else [] for p in parent]
        self.length = [self.length[p] if 0 <= p < seqs else 0 for p in parent]

    def grow(self, new):
        """(rows, positions, granted) for new[b] tokens each."""
        refs = self.refs()
        free = [p for p in range(self.P) if refs[p] == 0]
        asked, rows, positions, granted = 0, [], [], []
        for b, n in enumerate(new):
            old, pages = self.length[b], -(-(self.length[b] + n) // self.page)
            copy = int(n > 0 and old % self.page != 0 and refs[self.held[b][-1]] > 1)
            need = pages - len(self.held[b]) + copy if n else 0
            fits = n > 0 and pages <= self.W
            if fits:
                asked += need
                fits = need == 0 or asked <= len(free)
            if fits:
                take = free[asked - need: asked]
                if copy:
                    self.pool[:, take[0]] = self.pool[:, self.held[b][-1]]
                    self.held[b][-1] = take[0]
                self.held[b] += take[copy:]
                self.length[b] = old + n
            granted.append(n if fits else 0)
            for i in range(old, old + n):
                positions.append(i)
                rows.append(self.held[b][i // self.page] * self.page + i % self.page if fits else -1)
        return rows, positions, granted

    def compact(self):
        refs = self.refs()
        live = sum(r > 0 for r in refs)
        holes = [p for p in range(live) if refs[p] == 0]
        goes = dict(zip([p for p in range(live, self.P) if refs[p]], holes))
        for src, dst in goes.items():
            self.pool[:, dst] = self.pool[:, src]
        self.held = [[goes.get(p, p) for p in h] for h in self.held]
        return live


def int8(X, W, sx, sw, bias):
    """(y fp64, acc int64) of codes X [M, K], W [N, K]: fp64 products are exact (K * 2^14 < 2^53)."""
    acc = X.double() @ W.double().t()
    y = acc * (sx.double()[:, None] * sw.double()[None])
    return (y if bias is None else y + bias.double()), acc.long()
