"""bt_int8_pack at the most weights that it takes, N * K = 2^36: 64 GB, 2^32 pieces of 16 bytes."""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_pack_of_the_most_weights():
    N, K = 1 << 23, 1 << 13
    print(f"[gpu-case] int8 pack of {N} x {K}", flush=True)
    assert bt.int8_weight_bytes(N, K) == 1 << 36
    if torch.cuda.get_device_properties(0).total_memory < 160 << 30:
        pytest.skip("two arrays of 64 GB")
    W = torch.zeros((N, K), dtype=torch.int8, device=DEV)
    near = [0, 1, 15, 16, 4097, 1 << 22, N - 17, N - 1]
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for n in near:
        W[n] = torch.randint(-128, 128, (K,), generator=g, device=DEV, dtype=torch.int8)
    w = bt.pack_int8(W, torch.ones(N, device=DEV))
    blocks = w.data.view(torch.int8)[: 1 << 36].view(N // 16, K // 64, 4, 16, 16)
    for n in near:
        assert torch.equal(blocks[n // 16, :, :, n % 16].reshape(-1), W[n]), n
    # one row of the last sixteen holds more than zeros besides
    assert not bool(blocks[-1, :, :, :15].any()) and not bool(blocks[1 << 17].any())
    del W, blocks, w
    torch.cuda.empty_cache()
