"""A Cache4 whose pages hold another number of tokens than the Pages' is refused: the places that pages_grow gives would
name other tokens in it. Checked on the host before any launch."""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests.test_api_validation import host_ok  # noqa: F401  (fixture)


@pytest.mark.parametrize("tokens", [16, 32, 128])
def test_another_page_size_is_refused(host_ok, tokens):  # noqa: F811
    pages = bt.Pages(2, 3, 8, 64, device="cpu")
    cache = bt.Cache4(8, tokens, 2, 64, device="cpu")
    start = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match=f"pages of {tokens} tokens.*64"):
        bt.pages_grow(pages, start, cache, tokens=2)
    with pytest.raises(ValueError, match=f"pages of {tokens} tokens.*64"):
        bt.pages_compact(pages, cache)


def test_the_same_page_size_goes_on(host_ok):  # noqa: F811
    pages = bt.Pages(2, 3, 8, 64, device="cpu")
    with pytest.raises(AssertionError, match="bt_pages_grow was called"):  # the fixture's end of the way
        bt.pages_grow(pages, torch.zeros(3, dtype=torch.int32), bt.Cache4(8, 64, 2, 64, device="cpu"), tokens=2)
    # a tensor says nothing of tokens
    with pytest.raises(AssertionError, match="bt_pages_grow was called"):
        bt.pages_grow(pages, torch.zeros(3, dtype=torch.int32), torch.zeros((1, 8, 16), dtype=torch.uint8), tokens=2)
