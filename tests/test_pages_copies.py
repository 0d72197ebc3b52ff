"""Copies of a Pages: deep ones, pickled ones and saved ones have a state and a workspace of their own, and every call on
them goes there; shallow ones share the state. By the addresses that the calls hand to the library, so without a GPU."""
import copy
import io
import pickle

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from bit_ternary_weight_absmean_amd import cache as module

SEQS, W, P, PAGE = 3, 4, 8, 16


def saved(pages):
    f = io.BytesIO()
    torch.save(pages, f)
    f.seek(0)
    return torch.load(f, weights_only=False)  # what this test wrote


WAYS = {"deepcopy": copy.deepcopy, "pickle": lambda p: pickle.loads(pickle.dumps(p)), "save": saved}


@pytest.fixture
def calls(monkeypatch):
    """The (function, arguments) of the calls that would go to the library."""
    seen = []
    monkeypatch.setattr(module.api, "_on_device", lambda t: True)
    monkeypatch.setattr(module, "_call", lambda dev, fn, *args: seen.append((fn.__name__, args)))
    return seen


def make():
    pages = bt.Pages(SEQS, W, P, PAGE, device="cpu")
    pages.table[1, 0], pages.length[1], pages.refs[3], pages.first[0] = 3, 9, 1, 2
    return pages


def every_call(pages, calls, workspace=None):
    """The addresses (table, length, refs, first, workspace) that each call on `pages` gets."""
    del calls[:]
    pool, start = torch.zeros((1, P, 32), dtype=torch.uint8), torch.zeros(SEQS + 1, dtype=torch.int32)
    bt.pages_grow(pages, start, pool, tokens=5)
    bt.pages_fork(pages, torch.zeros(SEQS, dtype=torch.int32))
    bt.pages_compact(pages, pool)
    grow, fork, compact = (args for _, args in calls)
    assert compact[1] == grow[1] and compact[2:4] == grow[3:5] and fork[1:5] == grow[1:5]
    assert grow[-1] == fork[-1] == compact[-1]
    return (*grow[1:5], grow[-1])


def check(pages, got):
    """The addresses are those of the object's own arrays, which are views of its state."""
    at = pages.state.data_ptr()
    cells = SEQS * W
    assert got[:4] == (at, at + 4 * cells, at + 4 * (cells + SEQS), at + 4 * (cells + SEQS + P))
    assert got[:4] == tuple(t.data_ptr() for t in (pages.table, pages.length, pages.refs, pages.first))
    assert pages.table.shape == (SEQS, W) and pages.length.shape == (SEQS,) and pages.refs.shape == (P,)
    assert pages.device == pages.state.device


@pytest.mark.parametrize("way", WAYS)
def test_a_copy_has_its_own_arrays(calls, way):
    pages = make()
    before = every_call(pages, calls)
    check(pages, before)
    other = WAYS[way](pages)
    assert (other.seqs, other.max_pages, other.pages, other.page_tokens) == (SEQS, W, P, PAGE)
    assert torch.equal(other.state, pages.state)
    got = every_call(other, calls)
    check(other, got)
    size = 4 * pages.state.numel()
    assert abs(other.state.data_ptr() - pages.state.data_ptr()) >= size
    assert got[4] != before[4]  # the two may run at once
    # what is done to one shows in its own views, and not in the other
    other.state.zero_()
    assert not other.table.any() and not other.length.any() and not other.refs.any() and not other.first.any()
    assert pages.table[1, 0] == 3 and pages.length[1] == 9
    assert every_call(pages, calls) == before


def test_a_shallow_copy_shares_the_state(calls):
    pages = make()
    other = copy.copy(pages)
    got = every_call(other, calls)
    check(other, got)
    assert got[:4] == every_call(pages, calls)[:4]
    pages.length[0] = 7
    assert other.length[0] == 7


def test_a_copy_outlives_the_first(calls):
    pages = make()
    other = pickle.loads(pickle.dumps(copy.deepcopy(pages)))
    del pages
    check(other, every_call(other, calls))
    assert other.table[1].tolist() == [3, -1, -1, -1] and other.first.tolist() == [2]


@pytest.mark.gpu
@pytest.mark.parametrize("way", WAYS)
def test_a_copy_goes_its_own_way(way):
    """On the GPU: a copy made in the middle, both go on with other tokens and forks."""
    print(f"[gpu-case] pages copy by {way}", flush=True)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda:0")  # noqa: E731
    pages = bt.Pages(SEQS, W, P, PAGE, device="cuda:0")
    pool = torch.zeros((1, P, 16), dtype=torch.uint8, device="cuda:0")
    bt.pages_grow(pages, i32([0, 20, 25, 25]), pool, tokens=25)
    other = WAYS[way](pages)
    state = pages.state.clone()
    rows, _, _ = bt.pages_grow(other, i32([0, 0, 0, 17]), pool, tokens=17)
    assert rows.tolist() == list(range(48, 65))
    bt.pages_fork(other, i32([2, 1, 2]))
    bt.pages_compact(other, pool)
    assert torch.equal(pages.state, state)
    assert other.table.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1], [0, 1, -1, -1]]
    assert other.length.tolist() == [17, 5, 17] and other.refs.tolist() == [2, 2, 1, 0, 0, 0, 0, 0] and int(other.first) == 3
    rows, _, _ = bt.pages_grow(pages, i32([0, 1, 1, 1]), pool, tokens=1)
    assert rows.tolist() == [20] and pages.length.tolist() == [21, 5, 0]
