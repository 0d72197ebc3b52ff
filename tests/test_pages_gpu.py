"""The pages' bookkeeping (grow, fork, compact, copy) against a model that goes one sequence and page at a time: all
of the state and the pool's bytes are equal after every step."""
import random

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import cache_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return i32(out)


class Both:
    """The library and the model, side by side."""

    def __init__(self, seqs, W, pages, page, layers=2, page_bytes=48, seed=0):
        g = torch.Generator().manual_seed(seed)
        pool = torch.randint(0, 256, (layers, pages, page_bytes), generator=g, dtype=torch.uint8)
        self.pool = pool.to(DEV)
        self.pages = bt.Pages(seqs, W, pages, page, device=DEV)
        self.model = cache_ref.Model(seqs, W, pages, page, pool)

    def same(self):
        p, m = self.pages, self.model
        assert p.table.tolist() == m.table()
        assert p.length.tolist() == m.length
        refs = m.refs()
        assert p.refs.tolist() == refs
        assert torch.equal(self.pool.cpu(), m.pool)
        first = int(p.first)
        assert all(refs[:first]), "a page below `first` is free"

    def grow(self, new, tail=0):
        want = self.model.grow(new)
        total = sum(new)
        rows, positions, granted = bt.pages_grow(self.pages, starts(new), self.pool, tokens=total + tail)
        assert rows.tolist() == want[0] + [-1] * tail
        assert positions.tolist() == want[1] + [-1] * tail
        assert granted.tolist() == want[2]
        self.same()
        return want[2]

    def fork(self, parent):
        self.model.fork(parent)
        bt.pages_fork(self.pages, i32(parent))
        self.same()

    def compact(self):
        live = self.model.compact()
        bt.pages_compact(self.pages, self.pool)
        assert int(self.pages.first) == live
        self.same()


SHAPES = [
    # seqs, max_pages, pages, page_tokens, layers, page_bytes
    (1, 4, 5, 16, 1, 16),
    (5, 7, 20, 16, 2, 48),
    (17, 9, 60, 1, 3, 16),
    (40, 30, 300, 128, 1, 16400),
    (1500, 3, 5000, 4, 1, 16),
    (3, 700, 9001, 16, 1, 32),
]


@pytest.mark.parametrize("seqs,W,pages,page,layers,size", SHAPES)
def test_random_steps(seqs, W, pages, page, layers, size):
    note(f"pages {seqs} x {W} over {pages} of {page}, {layers} layers of {size}")
    r = random.Random(seqs * 1000 + page)
    both = Both(seqs, W, pages, page, layers, size, seed=page)
    refused = 0
    for turn in range(14):
        kind = r.choice(["decode", "prompt", "prompt", "fork", "beams", "end", "compact"])
        if turn == 0 or kind == "prompt":
            new = [r.choice([0, 1, page, r.randint(0, W * page // 2), r.randint(0, W * page + 3)]) for _ in range(seqs)]
            refused += sum(n > 0 and not got for n, got in zip(new, both.grow(new, tail=turn % 3)))
        elif kind == "decode":
            both.grow([r.choice([0, 1, 1, 1, 5]) for _ in range(seqs)])
        elif kind == "fork":
            both.fork([r.randrange(-1, seqs + 1) for _ in range(seqs)])
        elif kind == "beams":
            both.fork([min(seqs - 1, b // 4 * 4 + r.randrange(4)) for b in range(seqs)])
            both.grow([1] * seqs)
        elif kind == "end":
            both.fork([b if r.random() < 0.6 else -1 for b in range(seqs)])
        else:
            both.compact()
    both.fork([-1] * seqs)
    assert not any(both.model.refs())
    both.compact()
    note(f"refused {refused}")


def test_every_sharer_copies():
    """Four beams on one partly filled page: four copies, and the shared page is free after them."""
    note("sharers")
    both = Both(4, 4, 12, 16)
    both.grow([20, 0, 0, 0])
    both.fork([0, 0, 0, 0])
    both.grow([1, 1, 0, 1])
    assert both.model.refs()[1] == 1  # sequence 2 did not grow and keeps it
    both.grow([0, 0, 1, 0])
    both.fork([0, 0, 0, 0])
    both.grow([12, 12, 12, 12])  # fills the last page to its end
    both.fork([1, 1, 1, 1])
    both.grow([1, 1, 1, 1])  # a new page each: nothing to copy


def test_refused():
    """The pool is too small: a sequence that gets nothing leaves the state as it was, those without need go on, and
    those behind it that need pages wait."""
    note("refused")
    both = Both(5, 8, 6, 16)
    assert both.grow([16, 20, 1, 0, 0]) == [16, 20, 1, 0, 0]  # 4 pages
    assert both.grow([17, 1, 1, 1, 40]) == [17, 1, 1, 0, 0]  # 2 more for the first: none for the new ones
    assert both.grow([0, 0, 200, 1, 0]) == [0, 0, 0, 0, 0]  # past max_pages, and none left
    both.fork([-1, 1, 2, 3, 4])
    assert both.grow([0, 1, 1, 1, 33]) == [0, 1, 1, 1, 0]


def test_without_pool_and_with_a_cache():
    note("pools")
    pages = bt.Pages(2, 4, 8, 16, device=DEV)
    cache = bt.Cache4(8, 16, 2, 64, layers=3)
    cache.data.random_(0, 256)
    before = cache.data.clone()
    bt.pages_grow(pages, starts([20, 3]), cache, tokens=23)
    bt.pages_fork(pages, i32([0, 0]))
    bt.pages_grow(pages, starts([0, 1]), cache, tokens=1)  # page 2 was dropped by sequence 1 and becomes the copy
    assert torch.equal(cache.data[:, 2], before[:, 1]) and torch.equal(cache.data[:, :2], before[:, :2])
    assert pages.table.tolist() == [[0, 1, -1, -1], [0, 2, -1, -1]]
    empty = torch.empty((0, 8, 16), dtype=torch.uint8, device=DEV)
    bt.pages_grow(pages, starts([1, 1]), empty, tokens=2)
    none = bt.Pages(3, 2, 0, 16, device=DEV)
    _, _, granted = bt.pages_grow(none, starts([1, 0, 1]), torch.empty((1, 0, 16), dtype=torch.uint8, device=DEV), tokens=2)
    assert granted.tolist() == [0, 0, 0]
    bt.pages_compact(none, torch.empty((1, 0, 16), dtype=torch.uint8, device=DEV))
    bt.pages_fork(none, i32([2, 1, 0]))


def test_pages_copy():
    note("copy")
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for dtype, shape in ((torch.uint8, (3, 40, 20000)), (torch.bfloat16, (2, 40, 16, 2, 8)), (torch.float32, (1, 40, 4))):
        pool = torch.randint(0, 100, shape, generator=g, device=DEV).to(dtype)
        src, dst = [0, 5, -1, 40, 7, 9, 39], [1, 6, 8, 2, -3, 40, 38]
        want = pool.clone()
        for s, d in ((0, 1), (5, 6), (39, 38)):
            want[:, d] = pool[:, s]
        bt.pages_copy(pool, i32(src), i32(dst))
        assert torch.equal(pool, want)
        bt.pages_copy(pool, i32([]), i32([]))
        assert torch.equal(pool, want)


def test_far_pool():
    """Copies past 4 GiB of a pool of several layers."""
    layers, pages, size = 3, 90000, 16 * 1024 + 16
    note(f"far pool: {layers * pages * size} bytes")
    pool = torch.zeros((layers, pages, size), dtype=torch.uint8, device=DEV)
    p = bt.Pages(2, 4, pages, 16, device=DEV)
    p.refs[: pages - 2] = 1  # all but the last two are taken by others
    p.table[0, 0], p.length[0], p.refs[pages - 3] = pages - 3, 5, 1
    pool[:, pages - 3] = torch.arange(size, device=DEV).to(torch.uint8)
    bt.pages_fork(p, i32([0, 0]))
    bt.pages_grow(p, starts([0, 1]), pool, tokens=1)
    assert p.table[1].tolist() == [pages - 2, -1, -1, -1] and int(p.refs[pages - 3]) == 1
    assert torch.equal(pool[:, pages - 2], pool[:, pages - 3]) and not bool(pool[:, pages - 1].any())
    p.refs[7] = 0
    bt.pages_compact(p, pool)
    assert int(p.table[1, 0]) == 7 and torch.equal(pool[:, 7], pool[:, pages - 3]) and int(p.first) == pages - 2


def test_replays():
    """A captured step (fork, grow) replayed from the state it left, and a second graph with a workspace of its own."""
    note("replays")
    seqs = 6
    both = Both(seqs, 20, 100, 16, layers=2, page_bytes=64)
    both.grow([3, 17, 0, 40, 5, 64])
    parent, q_start = i32(list(range(seqs))), starts([1] * seqs)
    out = tuple(torch.empty(seqs, dtype=torch.int32, device=DEV) for _ in range(3))
    ws = torch.empty_like(both.pages._workspace)
    kept = both.pages.state.clone(), both.pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        bt.pages_fork(both.pages, parent, workspace=ws)
        bt.pages_grow(both.pages, q_start, both.pool, out=out, workspace=ws)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            bt.pages_fork(both.pages, parent, workspace=ws)
            bt.pages_grow(both.pages, q_start, both.pool, out=out, workspace=ws)
    torch.cuda.synchronize()
    both.pages.state.copy_(kept[0])
    both.pool.copy_(kept[1])
    r = random.Random(4)
    for _ in range(12):
        order = [r.randrange(-1, seqs) for _ in range(seqs)]
        parent.copy_(i32(order))
        graph.replay()
        both.model.fork(order)
        rows, positions, granted = both.model.grow([1] * seqs)
        assert out[0].tolist() == rows and out[1].tolist() == positions and out[2].tolist() == granted
        both.same()
        if r.random() < 0.3:
            both.compact()
