"""What the Python binding checks before a call reaches the library; no GPU needed."""
import ctypes

import pytest
import torch


@pytest.fixture
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


@pytest.mark.parametrize("device,want", [(None, 3), ("cuda", 3), (torch.device("cuda"), 3), ("cuda:1", 1), (0, 0), (2, 2),
                                         (torch.device("cuda", 0), 0)])
def test_a_handle_without_an_index_is_on_the_current_device(dattn, monkeypatch, device, want):
    seen = []

    def create(cfg, dev, out):
        seen.append(dev)
        return dattn.OK

    monkeypatch.setattr(dattn.lib, "dattn_create", create)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    h = dattn.Handle(8, 2, 128, [{"kind": dattn.CACHE_RING, "ring_slots": 4}], 1, device=device)
    assert seen == [want] and h.device == want
    h._h = ctypes.c_void_p()


def test_a_handle_is_not_on_the_host(dattn):
    with pytest.raises(ValueError):
        dattn.Handle(8, 2, 128, [{"kind": dattn.CACHE_RING, "ring_slots": 4}], 1, device="cpu")
