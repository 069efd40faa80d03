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


def test_4_bit_layers_are_paged_in_whole_blocks(dattn):
    """Refused before anything is allocated or launched."""
    def status(**layer):
        cfg = dattn.LayerConfig(layer.get("kind", dattn.CACHE_PAGED), layer.get("ring_slots", 0), layer.get("page_size", 16), 0, 0.0,
                                None, None, 0.0, layer.get("fmt", dattn.KV_INT4), 1.0, 1.0, layer.get("log_decay"))
        c = dattn.Config(8, 2, 128, 4, 64, 0, 1, ctypes.pointer(cfg), 0)
        return dattn.lib.dattn_create(ctypes.byref(c), 0, ctypes.byref(ctypes.c_void_p()))
    for page in (1, 8, 24, 100):
        assert status(page_size=page) == dattn.EUNSUPPORTED
    assert status(kind=dattn.CACHE_RING, ring_slots=64) == dattn.EUNSUPPORTED
    decay = (ctypes.c_float * 2)(0.0, 0.0)
    assert status(kind=dattn.CACHE_STATE, log_decay=ctypes.addressof(decay)) == dattn.EUNSUPPORTED
    assert status(fmt=3) == dattn.EINVAL and status(fmt=-1) == dattn.EINVAL
    assert dattn.lib.dattn_read_kv(None, 0, None, 1, 1, None, None, None, None, None) == dattn.EINVAL
    for page in (0, 8, 24):
        with pytest.raises(ValueError):
            dattn.int4_pool(4, 2, page, 128, device="cpu")
    assert dattn.int4_pool(4, 2, 48, 256, device="cpu").shape == (4, 2, 3 * 9 * 256)


def test_4_bit_pools_have_the_handles_shape(dattn, monkeypatch):
    monkeypatch.setattr(dattn, "_ptr", lambda t: None)
    monkeypatch.setattr(dattn.lib, "dattn_create", lambda cfg, dev, out: dattn.OK)
    h = dattn.Handle(8, 2, 128, [{"kind": dattn.CACHE_PAGED, "page_size": 32, "kv_format": dattn.KV_INT4}], 4, max_context=64, device=0)
    h._h = ctypes.c_void_p()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = lambda *s: dattn.int4_pool(*s, device="cpu")  # noqa: E731
    good, row = pool(9, 2, 32, 128), (i32(4, 4), i32(4))
    for k, v in ((pool(9, 1, 32, 128), good), (good, pool(9, 2, 16, 128)), (pool(9, 2, 32, 256), pool(9, 2, 32, 256)),
                 (good, good.to(torch.int8)), (bf(9, 2, 32, 128), bf(9, 2, 32, 128)), (good, pool(8, 2, 32, 128))):
        c = dattn.paged_cache(k, v, *row)
        for call in (lambda: h.decode(0, c, bf(4, 8, 128), bf(4, 2, 128), bf(4, 2, 128), i32(4), torch.zeros(4, 8, 128)),
                     lambda: h.append_kv(0, c, bf(4, 3, 2, 128), bf(4, 3, 2, 128), i32(4), i32(4), rotate=False),
                     lambda: h.read_kv(0, c, i32(4), i32(4), bf(4, 3, 2, 128), bf(4, 3, 2, 128))):
            with pytest.raises(ValueError):
                call()
    c = dattn.paged_cache(good, good.clone(), *row)
    out = bf(4, 3, 2, 128)
    for args in ((i32(4), i32(4), out.float(), out), (i32(4), i32(4), out, out[:, :2]), (i32(4), i32(4), bf(4, 3, 1, 128), bf(4, 3, 1, 128)),
                 (i32(4).long(), i32(4), out, out), (i32(4), i32(3), out, out), (i32(3), i32(4), out, out)):
        with pytest.raises(ValueError):
            h.read_kv(0, c, *args)


def test_4_bit_pools_stay_off_other_layers(dattn, monkeypatch):
    """(A bf16 layer would take their bytes for entries three to four times as long.)"""
    monkeypatch.setattr(dattn, "_ptr", lambda t: None)
    monkeypatch.setattr(dattn.lib, "dattn_create", lambda cfg, dev, out: dattn.OK)
    h = dattn.Handle(8, 2, 128, [{"kind": dattn.CACHE_PAGED, "page_size": 16},
                                 {"kind": dattn.CACHE_PAGED, "page_size": 16, "kv_format": dattn.KV_E4M3, "k_scale": 1.0, "v_scale": 1.0}],
                     4, max_context=64, max_verify_rows=3, device=0)
    h._h = ctypes.c_void_p()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool, row = dattn.int4_pool(9, 2, 16, 128, device="cpu"), (i32(4, 4), i32(4))
    c = dattn.paged_cache(pool, pool.clone(), *row)
    q, kv, out = bf(4, 3, 8, 128), bf(4, 3, 2, 128), torch.zeros(4, 3, 8, 128)
    summary = bf(9, 2, 128)
    one = (q[:, 0], kv[:, 0], kv[:, 0], i32(4), out[:, 0])
    for layer in (0, 1):
        for call in (lambda: h.decode(layer, c, *one), lambda: h.append_kv(layer, c, kv, kv, i32(4), i32(4), rotate=False),
                     lambda: h.read_kv(layer, c, i32(4), i32(4), kv, kv), lambda: h.sparse_decode(layer, c, summary, *one, 2),
                     lambda: h.summarize(layer, c, summary, i32(4), i32(4), 3), lambda: h.verify(layer, c, q, kv, kv, i32(4, 3), out),
                     lambda: h.commit(layer, c, kv, kv, i32(4, 3), i32(4, 3), i32(4), i32(4)),
                     lambda: h.prefill(layer, c, q, kv, kv, i32(4), i32(4), out)):
            with pytest.raises(ValueError, match="4-bit"):
                call()
    # (a byte pool of an E4M3 layer is none)
    e4m3 = torch.zeros(9, 2, 16, 128, dtype=torch.uint8)
    h._check_pools(1, dattn.paged_cache(e4m3, e4m3.clone(), *row))


def test_byte_pools_of_a_layers_own_pages_are_no_4_bit_pools(dattn, monkeypatch):
    """An E4M3 layer's bytes (or a bf16 layer's, viewed so) with a head's rows flat: as many as its pages have."""
    monkeypatch.setattr(dattn, "_ptr", lambda t: None)
    monkeypatch.setattr(dattn.lib, "dattn_create", lambda cfg, dev, out: dattn.OK)
    H, P, D = 2, 16, 128
    h = dattn.Handle(8, H, D, [{"kind": dattn.CACHE_PAGED, "page_size": P},
                               {"kind": dattn.CACHE_PAGED, "page_size": P, "kv_format": dattn.KV_E4M3, "k_scale": 1.0, "v_scale": 1.0}],
                     4, max_context=64, device=0)
    h._h = ctypes.c_void_p()
    row = torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for layer, size in ((0, 2), (1, 1)):
        for shape in ((9, H, P * D * size), (9, H * P, D * size), (9, H, P, D * size)):
            pool = torch.zeros(shape, dtype=torch.uint8)
            h._check_pools(layer, dattn.paged_cache(pool, pool.clone(), *row))
        for few in (P * D * size - 1, P // 16 * 9 * D, P * D * size + 16):
            pool = torch.zeros(9, H, few, dtype=torch.uint8)
            with pytest.raises(ValueError, match="4-bit"):
                h._check_pools(layer, dattn.paged_cache(pool, pool.clone(), *row))


def test_read_back_of_more_streams_than_the_cache_names(dattn, monkeypatch):
    monkeypatch.setattr(dattn, "_ptr", lambda t: None)
    monkeypatch.setattr(dattn.lib, "dattn_create", lambda cfg, dev, out: dattn.OK)
    monkeypatch.setattr(dattn.lib, "dattn_read_kv", lambda *a: dattn.OK)
    monkeypatch.setattr(dattn, "_stream_ptr", lambda stream, device=None: 0)
    H, P, D = 2, 16, 128
    h = dattn.Handle(8, H, D, [{"kind": dattn.CACHE_PAGED, "page_size": P}, {"kind": dattn.CACHE_RING, "ring_slots": 32},
                               {"kind": dattn.CACHE_PAGED, "page_size": P, "kv_format": dattn.KV_INT4}], 4, max_context=64, device=0)
    h._h = ctypes.c_void_p()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    four = [dattn.int4_pool(9, H, P, D, device="cpu") for _ in range(2)]
    caches = {0: [dattn.paged_cache(bf(9, H, P, D), bf(9, H, P, D), i32(3, 4), i32(1))],
              1: [dattn.ring_cache(bf(9, H, 32, D), bf(9, H, 32, D), i32(9), i32(9), i32(3))],
              2: [dattn.paged_cache(*four, i32(3, 4), i32(3))]}
    for layer, (cache,) in caches.items():
        h.read_kv(layer, cache, i32(3), i32(3), bf(3, 2, H, D), bf(3, 2, H, D))
        h.read_kv(layer, cache, i32(1), i32(1), bf(1, 2, H, D), bf(1, 2, H, D))
        with pytest.raises(ValueError, match="3 streams"):
            h.read_kv(layer, cache, i32(4), i32(4), bf(4, 2, H, D), bf(4, 2, H, D))
    # (rows named by their numbers: the library compares each with the pool's)
    h.read_kv(1, dattn.ring_cache(bf(9, H, 32, D), bf(9, H, 32, D), i32(1), i32(1)), i32(4), i32(4), bf(4, 2, H, D), bf(4, 2, H, D))
