"""The 4-bit cache as a server runs it, around the framework's own products: fused ternary QKV projection -> places
for the new tokens -> head norms and rotation -> write -> attention over the cache -> ternary O projection -> int8 head;
a prompt batch, a beam search's steps (fork, copies on write) captured in a graph, then requests that end and a
compaction. Each step is compared with the definition in 64 bits on the step's own inputs, with the operators' own
tolerances, and all of it with a run that keeps every sequence's keys apart."""
import random

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref, cache_ref
from tests.test_cache4_gpu import tolerance
from tests.test_int8_gpu import check as check_int8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Server:
    """Two layers of a 2B class attention block (hidden 2560, 20 query and 5 key heads of 128) and a head."""

    heads, kv, D, hidden, layers, vocab = 20, 5, 128, 2560, 2, 1000

    def __init__(self, seqs, max_pages, pages, page):
        g = torch.Generator(device=DEV)
        g.manual_seed(21)
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        wide = (self.heads + 2 * self.kv) * self.D
        self.wqkv = [bt.pack_weights(0.02 * rnd(wide, self.hidden)) for _ in range(self.layers)]
        self.wo = [bt.pack_weights(0.02 * rnd(self.hidden, self.heads * self.D)) for _ in range(self.layers)]
        self.head = bt.pack_weights_int8(0.02 * rnd(self.vocab, self.hidden))
        self.qw, self.kw = 1 + 0.1 * rnd(self.D), 1 + 0.1 * rnd(self.D)
        self.inv = bt.rope_frequencies(self.D, 500000.0, DEV)
        self.cache = bt.Cache4(pages, page, self.kv, self.D, layers=self.layers)
        self.pages = bt.Pages(seqs, max_pages, pages, page, device=DEV)

    def buffers(self, T):
        e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
        q = e(T, self.heads, self.D, dtype=torch.bfloat16)
        kv = [[e(T, self.kv, self.D, dtype=torch.bfloat16) for _ in range(2)] for _ in range(self.layers)]
        return {"q": [q, torch.empty_like(q)], "kv": kv, "grown": tuple(e(n, dtype=torch.int32) for n in (T, T, self.pages.seqs)),
                "o": [e(T, self.heads, self.D) for _ in range(self.layers)], "y": [e(T, self.hidden) for _ in range(self.layers)],
                "lse": [e(T, self.heads) for _ in range(self.layers)], "logits": e(T, self.vocab, dtype=torch.bfloat16)}

    def step(self, x, q_start, b, parent=None):
        if parent is not None:
            bt.pages_fork(self.pages, parent)
        rows, positions, _ = bt.pages_grow(self.pages, q_start, self.cache, out=b["grown"])
        for i in range(self.layers):
            qkv, _ = bt.linear(x, self.wqkv[i])
            q, (k, v) = b["q"][i], b["kv"][i]
            bt.qk_norm_rope(qkv, positions, self.inv, self.heads, self.kv, self.qw, self.kw, out=(q, k, v))
            bt.cache4_write(self.cache, k, v, rows, layer=i)
            bt.attention4(q, self.cache, self.pages.table, self.pages.length, q_start, layer=i, out=b["o"][i], lse=b["lse"][i])
            bt.linear(b["o"][i].view(len(x), -1), self.wo[i], out_y=b["y"][i])
            x = b["y"][i]
        bt.int8_gemm(self.head, bt.quant_act(x), out=b["logits"])


class Kept:
    """Every sequence's cached values, as the write rounds them, kept apart."""

    def __init__(self, server, seqs):
        self.s, self.seqs = server, [[[], []] for _ in range(seqs)]

    def fork(self, parent):
        self.seqs = [[list(layer) for layer in self.seqs[p]] if 0 <= p < len(parent) else [[], []] for p in parent]

    def check(self, q_start, b):
        s = self.s
        for i in range(s.layers):
            rounded = [cache_ref.decode(*cache_ref.encode(t), s.D) for t in b["kv"][i]]
            for n, seq in enumerate(self.seqs):
                seq[i] += [(rounded[0][t], rounded[1][t]) for t in range(q_start[n], q_start[n + 1])]
            k_len = [len(seq[i]) for seq in self.seqs]
            k, v = (torch.stack([kv[j] for seq in self.seqs for kv in seq[i]]) for j in range(2))
            start = [sum(k_len[:n]) for n in range(len(k_len))]
            args = (q_start, start, k_len, True)
            q, out = b["q"][i], b["o"][i]
            ref, rlse = block_ref.attention(q.double(), k, v, *args)
            mag, _ = block_ref.attention(q.double(), k, v.abs(), *args)
            tol, ltol = tolerance(q, k, max(k_len), mag, ref, rlse, out.dtype)
            assert bool(((out.double() - ref).abs() <= tol).all())
            assert bool(((b["lse"][i].double() - rlse).abs() <= ltol).all())
            assert s.pages.length.tolist() == k_len
        xq, sx, _ = bt.quant_act(b["y"][-1])
        wq = self.head_codes()
        ref, acc = cache_ref.int8(xq[:, : s.hidden], wq, sx, s.head.scale, None)
        check_int8(b["logits"], ref, acc, sx, s.head.scale, None)

    def head_codes(self):
        s = self.s
        data = s.head.data.view(torch.int8)[: bt.int8_weight_bytes(s.vocab, s.hidden)]
        blocks = data.view(-1, s.hidden // 64, 4, 16, 16)
        return blocks.permute(0, 3, 1, 2, 4).reshape(-1, s.hidden)[: s.vocab]


def starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("page", [16, 64])
def test_prompts_beams_and_compaction(page):
    note(f"cache run, pages of {page}")
    seqs = 6
    s = Server(seqs, -(-400 // page), 3000 // page, page)
    kept = Kept(s, seqs)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    # two prompts, the second behind them continued
    for new in ([130, 45, 0, 0, 0, 0], [1, 200, 0, 0, 17, 0]):
        q_start = starts(new)
        b = s.buffers(q_start[-1])
        s.step(torch.randn(q_start[-1], s.hidden, generator=g, device=DEV), i32(q_start), b)
        kept.check(q_start, b)
    # beams of both prompts: a captured step, replayed with other parents and tokens
    q_start = starts([1] * seqs)
    b, x = s.buffers(seqs), torch.zeros(seqs, s.hidden, device=DEV)
    parent, qs = i32([0, 1, 0, 1, 0, 1]), i32(q_start)
    state, data = s.pages.state.clone(), s.cache.data.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step(x, qs, b, parent)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            s.step(x, qs, b, parent)
    torch.cuda.synchronize()
    s.pages.state.copy_(state)
    s.cache.data.copy_(data)
    r = random.Random(page)
    order = [0, 1, 0, 1, 0, 1]
    for turn in range(9):
        parent.copy_(i32(order))
        x.copy_(torch.randn(seqs, s.hidden, generator=g, device=DEV))
        graph.replay()
        kept.fork(order)
        kept.check(q_start, b)
        order = [r.choice([n, r.randrange(seqs)]) for n in range(seqs)]
    # three requests end, the rest go on behind a compaction
    order = [0, -1, 2, -1, -1, 5]
    bt.pages_fork(s.pages, i32(order))
    kept.fork(order)
    bt.pages_compact(s.pages, s.cache)
    live = int(s.pages.first)
    assert int((s.pages.refs > 0).sum()) == live and bool((s.pages.refs[:live] > 0).all())
    s.cache.data[:, live:] = 255  # handed back
    new = [1, 30, 1, 0, 0, 1]
    q_start = starts(new)
    b = s.buffers(q_start[-1])
    s.step(torch.randn(q_start[-1], s.hidden, generator=g, device=DEV), i32(q_start), b)
    kept.check(q_start, b)


def test_cached_prefix_for_the_16_bit_attention():
    """A prompt read back from the 4-bit cache as the shared prefix of bt_attention: the same as attention4 over both."""
    note("prefix read back")
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    page, kv, D, P, n = 32, 2, 64, 100, 7
    cache = bt.Cache4(8, page, kv, D)
    k, v = (torch.randn(P + n, kv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    bt.cache4_write(cache, k, v, i32(list(range(P + n))))
    kk, vv = bt.cache4_read(cache, i32(list(range(P + n))))
    q = torch.randn(n, 8, D, generator=g, device=DEV).bfloat16()
    a, _ = bt.attention4(q, cache, i32([[0, 1, 2, 3]]), i32([P + n]), i32([0, n]), out_dtype=torch.float32)
    b, _ = bt.attention(q, kk[P:], vv[P:], i32([0, n]), i32([0]), i32([n]), prefix_k=kk[:P], prefix_v=vv[:P],
                        out_dtype=torch.float32)
    args = ([0, n], [0], [P + n], True)
    ref, rlse = block_ref.attention(q.double(), kk.double(), vv.double(), *args)
    mag, _ = block_ref.attention(q.double(), kk.double(), vv.double().abs(), *args)
    tol, _ = tolerance(q, kk.double(), P + n, mag, ref, rlse, a.dtype)
    assert bool(((a.double() - ref).abs() <= tol).all())
    # bt_attention carries probabilities in two bf16 parts, 2^-16, of the sequence and of the prefix
    assert bool(((a.double() - b.double()).abs() <= 2 * tol + 2 * 2.0 ** -16 * mag).all())
