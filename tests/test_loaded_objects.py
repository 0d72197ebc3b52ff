"""A Cache4 or LoraAdapters that was saved on one device and loaded onto another goes by where its arrays are now: calls
with arrays of the device it came from are refused, and on the host nothing is launched."""
import io
import pickle

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from bit_ternary_weight_absmean_amd import api, cache as module

GPU = torch.device("cuda", 0)


def from_gpu(thing, *names):
    """`thing` (on the host) as it is when it was saved on a GPU and loaded here."""
    for name in names:
        object.__setattr__(thing, name, GPU)
    return pickle.loads(pickle.dumps(thing))


@pytest.fixture
def host(monkeypatch):
    """Lets host tensors through the checks; what would be called is noted with its device."""
    seen = []
    monkeypatch.setattr(api, "_on_device", lambda t: True)
    for where in (api, module):
        monkeypatch.setattr(where, "_call", lambda dev, fn, *args: seen.append(dev))
    return seen


def test_cache4(host):
    c = from_gpu(bt.Cache4(4, 16, 2, 64, layers=2, device="cpu"), "device")
    assert c.device == c.data.device == torch.device("cpu") and c.layers == 2
    k, rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    bt.cache4_write(c, k, k, rows, layer=1)
    bt.cache4_read(c, rows)
    bt.attention4(k, c, rows.view(1, 3), rows[:1], rows[:2])
    assert host == [torch.device("cpu")] * 3


def test_adapters(host):
    a = bt.LoraAdapters(torch.zeros((2, 4, 32)), torch.zeros((2, 8, 4)), torch.ones(2))
    a = from_gpu(a, "_dev")
    bt.lora_apply(torch.zeros((3, 32)), a, torch.zeros(3, dtype=torch.int32))
    assert host == [torch.device("cpu")]


def save(thing):
    f = io.BytesIO()
    torch.save(thing, f)
    return f


def load(f, where):
    f.seek(0)
    return torch.load(f, map_location=where, weights_only=False)  # what this test wrote


@pytest.mark.gpu
def test_loaded_onto_the_host_and_back():
    print("[gpu-case] loaded objects", flush=True)
    g = torch.Generator(device=GPU)
    g.manual_seed(1)
    k = torch.randn(3, 2, 64, generator=g, device=GPU).bfloat16()
    rows = torch.tensor([5, 17, 40], dtype=torch.int32, device=GPU)
    c = bt.Cache4(4, 16, 2, 64)
    bt.cache4_write(c, k, k, rows)
    f = save(c)
    host = load(f, "cpu")
    assert host.device == torch.device("cpu")
    for where in (GPU, torch.device("cpu")):  # the first: arrays on two devices; the second: no device at all
        with pytest.raises(ValueError):
            bt.cache4_write(host, k.to(where), k.to(where), rows.to(where))
        with pytest.raises(ValueError):
            bt.cache4_read(host, rows.to(where))
    back = load(f, GPU)
    for x, y in zip(bt.cache4_read(back, rows), bt.cache4_read(c, rows)):
        assert torch.equal(x, y)
    A, B = torch.randn(2, 4, 32, generator=g, device=GPU), torch.randn(2, 8, 4, generator=g, device=GPU)
    a = bt.LoraAdapters(A, B, torch.ones(2, device=GPU))
    X, index = torch.randn(3, 32, generator=g, device=GPU), torch.tensor([0, 1, -1], dtype=torch.int32, device=GPU)
    want, f = bt.lora_apply(X, a, index), save(a)
    host = load(f, "cpu")
    for where in (GPU, torch.device("cpu")):
        with pytest.raises(ValueError):
            bt.lora_apply(X.to(where), host, index.to(where))
    assert torch.equal(bt.lora_apply(X, load(f, GPU), index), want)
