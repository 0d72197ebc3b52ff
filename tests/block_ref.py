"""The attention-block operators' definitions in 64 bits (torch, any device), for the tests."""
import math

import torch


def lora(X, A, B, scale, index, base=None, ranks=None, group_rows=None):
    """(Y, magnitude): the result and the sum of the absolute values of its terms."""
    L, N, R = B.shape
    groups = list(group_rows) if group_rows is not None else [N]
    M = X.shape[0]
    y = torch.zeros((M, N), dtype=torch.float64, device=X.device) if base is None else base.double().clone()
    mag = y.abs()
    for m, a in enumerate(index.tolist()):
        if not 0 <= a < L:
            continue
        r = R if ranks is None else max(0, min(R, int(ranks[a])))
        col = 0
        for g, rows in enumerate(groups):
            down = A[a, g * R: g * R + r].double()
            up = B[a, col: col + rows, :r].double()
            x = X[m].double()
            s = scale[a].double()
            y[m, col: col + rows] += s * (up @ (down @ x))
            mag[m, col: col + rows] += s.abs() * (up.abs() @ (down.abs() @ x.abs()))
            col += rows
    return y, mag


def norm_rope(x, weight, eps, angle, rot, interleaved):
    """(y, magnitude) of heads x [M, H, D]; angle [M, rot / 2] fp64 or None."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
    y, mag = x.clone(), x.abs()
    if rot:
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = x[..., lo].clone(), x[..., hi].clone()
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        both = a.abs() + b.abs()
        mag[..., lo], mag[..., hi] = both, both
    return y, mag


def attention(q, k, v, q_start, k_start, k_len, causal, scale=None, prefix_k=None, prefix_v=None):
    """(out, lse) [T, Hq, D], [T, Hq] of the covered rows, from lists of offsets; rows behind the last
    sequence are NaN here. Only visible keys and values are read."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=q.device)
    for b in range(len(k_len)):
        lo, hi = q_start[b], q_start[b + 1]
        n, nk = hi - lo, k_len[b]
        if n == 0:
            continue
        ks, vs = k[k_start[b]: k_start[b] + nk].double(), v[k_start[b]: k_start[b] + nk].double()
        sees = torch.ones((n, nk), dtype=torch.bool, device=q.device)
        if causal:
            sees = torch.arange(nk, device=q.device)[None] <= (nk - n + torch.arange(n, device=q.device))[:, None]
        P = 0
        if prefix_k is not None:
            P = prefix_k.shape[0]
            ks, vs = torch.cat([prefix_k.double(), ks]), torch.cat([prefix_v.double(), vs])
            sees = torch.cat([torch.ones((n, P), dtype=torch.bool, device=q.device), sees], 1)
        ks, vs = ks.repeat_interleave(G, 1), vs.repeat_interleave(G, 1)  # [keys, Hq, D]
        s = torch.matmul(q[lo:hi].double().transpose(0, 1), ks.permute(1, 2, 0)) * scale
        s = torch.where(sees, s, torch.full_like(s, -math.inf))
        if s.shape[-1]:
            lse[lo:hi] = torch.logsumexp(s, -1).t()
            p = torch.exp(s - torch.logsumexp(s, -1, keepdim=True)).nan_to_num(nan=0.0)
        else:
            lse[lo:hi] = -math.inf
            p = s
        # a value reaches a row only where the row sees it
        fine = torch.isfinite(vs)
        o = torch.matmul(p, torch.where(fine, vs, torch.zeros_like(vs)).transpose(0, 1))
        if not bool(fine.all()):
            see = sees.double()[None].expand(Hq, -1, -1)
            for bad, value in ((vs == math.inf, math.inf), (vs == -math.inf, -math.inf), (vs.isnan(), math.nan)):
                hit = torch.matmul(see, bad.double().transpose(0, 1)) > 0
                o = o + torch.where(hit, torch.full_like(o, value), torch.zeros_like(o))
        out[lo:hi] = o.transpose(0, 1)
    return out, lse
