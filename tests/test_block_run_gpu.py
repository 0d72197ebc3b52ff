"""The attention block as a model runs it, around the framework's own products: fused QKV projection with
the requests' adapters -> head norms and rotation into the cache -> attention -> O projection, for a
prompt batch, then decode steps captured in a graph, and behind a shared prefix. Each step is compared
with the definition in 64 bits on the step's own inputs (their tolerances are the operators' own, given
with their tests), and the cached run with the uncached one."""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from bit_ternary_weight_absmean_amd import synth
from tests import block_ref
from tests.test_block_heads_gpu import close as close_heads
from tests.test_block_lora_gpu import close as close_lora

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


class Block:
    """One 2B class attention block: hidden 2560, 20 query and 5 key heads of 128, row-group scales."""

    heads, kv, D, hidden = 20, 5, 128, 2560

    def __init__(self, requests, slab, adapters=True):
        g = torch.Generator(device=DEV)
        g.manual_seed(77)
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        groups = synth.row_groups(synth.CFG_2B_DECODE, "qkv", 3840)
        self.wqkv = bt.pack_weights_rows(0.02 * rnd(3840, self.hidden), group_rows=groups)
        self.wo = bt.pack_weights(0.02 * rnd(self.hidden, self.hidden))
        self.qw, self.kw = 1 + 0.1 * rnd(self.D), 1 + 0.1 * rnd(self.D)
        self.inv = bt.rope_frequencies(self.D, 500000.0, DEV)
        L, R = 3, 8
        self.ad = bt.LoraAdapters((rnd(L, 3 * R, self.hidden) / 50).bfloat16(), rnd(L, 3840, R).bfloat16(),
                                  torch.rand(L, generator=g, device=DEV), group_rows=groups) if adapters else None
        self.k = torch.zeros((requests * slab, self.kv, self.D), dtype=torch.bfloat16, device=DEV)
        self.v = torch.zeros_like(self.k)
        self.slab = slab

    def step(self, X, index, pos, rows, q_start, k_start, k_len, out, prefix=(None, None)):
        qkv, _ = bt.linear(X, self.wqkv, adapters=self.ad, adapter_index=index)
        q = torch.empty((X.shape[0], self.heads, self.D), dtype=torch.bfloat16, device=DEV)
        bt.qk_norm_rope(qkv, pos, self.inv, self.heads, self.kv, self.qw, self.kw, rows=rows, out=(q, self.k, self.v))
        o, _ = bt.attention(q, self.k, self.v, q_start, k_start, k_len, prefix_k=prefix[0], prefix_v=prefix[1],
                            out_dtype=torch.float32)
        bt.linear(o.view(X.shape[0], -1), self.wo, out_y=out)
        return qkv, q, o


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def close_attention(o, q, k, v, q_start, k_start, k_len, pk=None, pv=None):
    args = (q_start, k_start, k_len, True)
    ref, _ = block_ref.attention(q, k, v, *args, prefix_k=pk, prefix_v=pv)
    mag, _ = block_ref.attention(q, k, v.abs(), *args, prefix_k=pk, prefix_v=None if pv is None else pv.abs())
    # scores here stay below 128 * 1.5^2 / sqrt(128) < 32: D / 8 + 2 sums of 2^-24, twice
    tol = (2 * 18 * 32 * 2.0 ** -24 + 2.0 ** -16 + 2.0 ** -17) * mag + 2.0 ** -24 * ref.abs()
    assert bool(((o.double() - ref).abs() <= tol).all()), float(((o.double() - ref).abs() / tol).max())


def test_prompts_then_decode_steps():
    note("block: prompts, then captured decode steps")
    lens, slab, steps = [37, 1, 90, 12], 128, 5
    n = len(lens)
    blk = Block(n, slab)
    total = [m + steps for m in lens]
    T = sum(lens)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    stream = [torch.randn((t, blk.hidden), generator=g, device=DEV) for t in total]
    index = i32([0, 2, -1, 1])
    starts = [0]
    for m in lens:
        starts.append(starts[-1] + m)
    k_start = i32([b * slab for b in range(n)])
    X = torch.cat([s[:m] for s, m in zip(stream, lens)])
    pos = torch.cat([torch.arange(m, device=DEV, dtype=torch.int32) for m in lens])
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(lens, device=DEV))
    rows = (seq * slab).to(torch.int32) + pos
    out = torch.empty_like(X)
    qkv, q, o = blk.step(X, index[seq], pos, rows, i32(starts), k_start, i32(lens), out)

    # every operator on its own inputs
    base, _ = bt.linear(X, blk.wqkv)
    ref, mag = block_ref.lora(X, blk.ad.A, blk.ad.B, blk.ad.scale, index[seq], base, None, blk.ad.group_rows)
    close_lora(qkv, ref, mag, blk.hidden, blk.ad.rank)
    heads = qkv.double().view(T, -1, blk.D)
    angle = pos.double()[:, None] * blk.inv
    close_heads(q, *block_ref.norm_rope(heads[:, :20], blk.qw, 1e-6, angle, 128, False))
    close_heads(blk.k[rows.long()], *block_ref.norm_rope(heads[:, 20:25], blk.kw, 1e-6, angle, 128, False))
    close_attention(o, q, blk.k, blk.v, starts, k_start.tolist(), lens)
    assert torch.equal(out, bt.linear(o.view(T, -1), blk.wo)[0])

    # decode: one token of each request per step, captured once and replayed
    x, dpos, drows = torch.zeros((n, blk.hidden), device=DEV), i32([0] * n), i32([-1] * n)
    dlen, dout, dq = i32(lens), torch.empty((n, blk.hidden), device=DEV), torch.arange(n + 1, device=DEV, dtype=torch.int32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        blk.step(x, index, dpos, drows, dq, k_start, dlen, dout)  # rows -1: writes nothing
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kept = blk.step(x, index, dpos, drows, dq, k_start, dlen, dout)
    for t in range(steps):
        at = torch.tensor(lens, device=DEV) + t
        x.copy_(torch.stack([stream[b][lens[b] + t] for b in range(n)]))
        dpos.copy_(at)
        drows.copy_(k_start + at)
        dlen.copy_(at + 1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = [m + t + 1 for m in lens]
        close_attention(kept[2], kept[1], blk.k, blk.v, list(range(n + 1)), k_start.tolist(), now)
        eager = torch.empty_like(dout)
        blk.step(x, index, dpos, drows, dq, k_start, dlen, eager)
        torch.cuda.synchronize()
        assert torch.equal(dout, eager), t

    # the same tokens as whole prompts: the cache holds the same rows up to the rounding of the products
    # (a token's product may run on another kernel, whose Y differs in its last bits)
    again = Block(n, slab)
    again.ad = blk.ad
    Xa = torch.cat(stream)
    pa = torch.cat([torch.arange(m, device=DEV, dtype=torch.int32) for m in total])
    sa = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(total, device=DEV))
    qs = [0]
    for m in total:
        qs.append(qs[-1] + m)
    again.step(Xa, index[sa], pa, (sa * slab).to(torch.int32) + pa, i32(qs), k_start, i32(total), torch.empty_like(Xa))
    step = torch.finfo(torch.bfloat16).eps
    for x1, x2 in ((blk.k, again.k), (blk.v, again.v)):
        assert bool(((x1.float() - x2.float()).abs() <= step * x1.float().abs() + 1e-4).all())


def test_batch_behind_a_shared_prefix():
    note("block: decode behind a shared prefix")
    n, slab, P = 6, 16, 300
    blk = Block(n, slab, adapters=False)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    prompt = torch.randn((P, blk.hidden), generator=g, device=DEV)
    qkv, _ = bt.linear(prompt, blk.wqkv)
    _, pk, pv = bt.qk_norm_rope(qkv, torch.arange(P, device=DEV, dtype=torch.int32), blk.inv, blk.heads, blk.kv, blk.qw,
                                blk.kw)
    own = [0, 3, 1, 15, 7, 0]
    blk.k.normal_()
    blk.v.normal_()
    x = torch.randn((n, blk.hidden), generator=g, device=DEV)
    pos = i32([P + m for m in own])
    k_start = i32([b * slab for b in range(n)])
    out = torch.empty((n, blk.hidden), device=DEV)
    q_start = torch.arange(n + 1, device=DEV, dtype=torch.int32)
    _, q, o = blk.step(x, None, pos, k_start + i32(own), q_start, k_start, i32([m + 1 for m in own]), out, (pk, pv))
    close_attention(o, q, blk.k, blk.v, list(range(n + 1)), k_start.tolist(), [m + 1 for m in own], pk, pv)
    # the same keys, each request with its own copy of the prefix
    k_all = torch.cat([torch.cat([pk, blk.k[b * slab: b * slab + own[b] + 1]]) for b in range(n)])
    v_all = torch.cat([torch.cat([pv, blk.v[b * slab: b * slab + own[b] + 1]]) for b in range(n)])
    lens = [P + m + 1 for m in own]
    first = [sum(lens[:b]) for b in range(n)]
    close_attention(o, q, k_all, v_all, list(range(n + 1)), first, lens)
    assert torch.equal(out, bt.linear(o.view(n, -1), blk.wo)[0])
