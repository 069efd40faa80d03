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


@pytest.fixture
def handle(dattn, monkeypatch):
    """A handle with a paged and a state layer that never reaches the library."""
    monkeypatch.setattr(dattn.lib, "dattn_create", lambda cfg, dev, out: dattn.OK)
    layers = [{"kind": dattn.CACHE_PAGED, "page_size": 16}, {"kind": dattn.CACHE_STATE, "log_decay": [0.0, -1.0]}]
    h = dattn.Handle(8, 2, 128, layers, 4, max_context=64, device=0, max_selected_pages=4)
    yield h
    h._h = ctypes.c_void_p()


def test_states_have_the_handles_shape(dattn, handle, monkeypatch):
    monkeypatch.setattr(dattn, "_ptr", lambda t: None)  # (host tensors stand in)
    with pytest.raises(TypeError):
        dattn.state_cache(torch.zeros(4, 2, 128, 128, dtype=torch.bfloat16))
    for shape in ((4, 2, 128), (4, 2, 128, 64), (4, 2, 2, 128, 128)):
        with pytest.raises(ValueError):
            dattn.state_cache(torch.zeros(shape))
    with pytest.raises(TypeError):
        dattn.state_cache(torch.zeros(4, 2, 128, 128), torch.zeros(4, dtype=torch.int64))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    paged = dattn.paged_cache(bf(4, 2, 16, 128), bf(4, 2, 16, 128), i32(4, 4), i32(4))
    for cache in (dattn.state_cache(torch.zeros(4, 1, 128, 128)), dattn.state_cache(torch.zeros(4, 2, 64, 64)),
                  dattn.state_cache(torch.zeros(4, 2, 128, 128), i32(3)), paged):
        with pytest.raises(ValueError):
            handle.decode(1, cache, bf(4, 8, 128), bf(4, 2, 128), bf(4, 2, 128), i32(4), torch.zeros(4, 8, 128))
        with pytest.raises(ValueError):
            handle.prefill(1, cache, bf(4, 3, 8, 128), bf(4, 3, 2, 128), bf(4, 3, 2, 128), i32(4), i32(4),
                           torch.zeros(4, 3, 8, 128))


def test_summaries_have_the_caches_shape(dattn, handle, monkeypatch):
    monkeypatch.setattr(dattn, "_ptr", lambda t: None)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = dattn.paged_cache(bf(9, 2, 16, 128), bf(9, 2, 16, 128), i32(4, 4), i32(4))
    x = (bf(4, 8, 128), bf(4, 2, 128), bf(4, 2, 128), i32(4), torch.zeros(4, 8, 128), 4)
    for summary, error in ((torch.zeros(9, 2, 128), TypeError), (bf(8, 2, 128), ValueError), (bf(9, 1, 128), ValueError),
                           (bf(9, 2, 64), ValueError), (bf(9 * 2 * 128), ValueError)):
        with pytest.raises(error):
            handle.sparse_decode(0, cache, summary, *x)
        with pytest.raises(error):
            handle.summarize(0, cache, summary, i32(4), i32(4), 16)
    for start, count in ((torch.zeros(4, dtype=torch.int64), i32(4)), (i32(4), torch.zeros(4)), (i32(4), i32(3))):
        with pytest.raises(ValueError):
            handle.summarize(0, cache, bf(9, 2, 128), start, count, 16)
