"""Entries of a table that name no page of the pool: bt_pages_grow leaves them alone, and tokens that would lie in such a
page have no place (-1), whatever the entry's bits shifted by the page's size would be."""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# Places are filled in by the one workgroup that plans (few tokens, few sequences), or by the launch behind it (more
# than 2048 tokens, or more than 1024 sequences).
@pytest.mark.parametrize("seqs,tail", [(3, 0), (3, 3000), (1100, 0)])
@pytest.mark.parametrize("entry", [-1, -(2 ** 31), 6, 2 ** 22 + 3, 2 ** 31 - 1])
def test_a_last_page_outside_the_pool(seqs, tail, entry):
    print(f"[gpu-case] pages entry {entry}, {seqs} sequences, {tail} tokens behind", flush=True)
    page, P, W = 1024, 6, 3
    pages = bt.Pages(seqs, W, P, page, device=DEV)
    pool = torch.zeros((1, P, 16), dtype=torch.uint8, device=DEV)
    # sequence 0: 10 tokens in page 0; sequence 1: 10 in a page that is none; sequence 2: nothing yet
    pages.table[0, 0], pages.length[0], pages.refs[0] = 0, 10, 1
    pages.table[1, 0], pages.length[1] = entry, 10
    start = [0, 2, 4, 6] + [6] * (seqs - 3)
    rows, positions, granted = bt.pages_grow(pages, i32(start), pool, tokens=6 + tail)
    assert granted.tolist() == [2, 2, 2] + [0] * (seqs - 3)
    assert rows.tolist() == [10, 11, -1, -1, page, page + 1] + [-1] * tail
    assert positions.tolist() == [10, 11, 10, 11, 0, 1] + [-1] * tail
    assert pages.table[:3].tolist() == [[0, -1, -1], [entry, -1, -1], [1, -1, -1]]
    assert pages.refs.tolist() == [1, 1, 0, 0, 0, 0]
    # past the page's end the tokens get a page of the pool
    rows, _, granted = bt.pages_grow(pages, i32([0, 0] + [1014] * (seqs - 1)), pool, tokens=1014)
    assert granted.tolist() == [0, 1014] + [0] * (seqs - 2)
    assert rows.tolist() == [-1] * 1012 + [2 * page, 2 * page + 1]
