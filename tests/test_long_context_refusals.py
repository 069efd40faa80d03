"""Host-side checks of the long-context entry points that answer without a GPU."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def create(dattn, layer, max_context=0, max_selected=0):
    layers = (dattn.LayerConfig * 1)(layer)
    cfg = dattn.Config(8, 2, 128, 1, max_context, 0, 1, layers, max_selected)
    h = ctypes.c_void_p()
    return dattn.lib.dattn_create(ctypes.byref(cfg), 0, ctypes.byref(h))


def state(dattn, decay, rotary=0, fmt=0, norm=None):
    d = None if decay is None else np.asarray(decay, np.float32)
    layer = dattn.LayerConfig(dattn.CACHE_STATE, 0, 0, rotary, 1e4, norm, None, 0.0, fmt, 1.0, 1.0,
                              None if d is None else d.ctypes.data)
    return layer, d


@pytest.mark.parametrize("decay", [None, [0.0, 0.1], [float("nan"), 0.0], [0.0, -np.inf]])
def test_decays_that_are_none(dattn, decay):
    layer, keep = state(dattn, decay)
    assert create(dattn, layer) == dattn.EINVAL


def test_state_layers_take_no_rotation_norm_or_fp8(dattn):
    w = np.zeros(128, np.uint16)
    for kw in ({"rotary": 64}, {"fmt": dattn.KV_E4M3}, {"norm": w.ctypes.data}):
        layer, keep = state(dattn, [0.0, -1.0], **kw)
        assert create(dattn, layer) == dattn.EUNSUPPORTED


def test_selection_limits(dattn):
    paged = dattn.LayerConfig(dattn.CACHE_PAGED, 0, 16, 0, 0.0, None, None, 0.0, 0, 1.0, 1.0, None)
    assert create(dattn, paged, 1000, -1) == dattn.EINVAL
    one = dattn.LayerConfig(dattn.CACHE_PAGED, 0, 1, 0, 0.0, None, None, 0.0, 0, 1.0, 1.0, None)
    assert create(dattn, one, 2 ** 31 - 1, 8) == dattn.EUNSUPPORTED  # a bitmap of so many pages does not fit


def test_null_arguments(dattn):
    lib = dattn.lib
    sel = dattn.PageSelection(None, 1, 0, 1, None)
    assert lib.dattn_sparse_decode(None, 0, None, None, ctypes.byref(sel), None) == dattn.EINVAL
    assert lib.dattn_sparse_decode(None, 0, None, None, None, None) == dattn.EINVAL
    assert lib.dattn_summarize(None, 0, None, None, 1, 1, None, None, None) == dattn.EINVAL


def test_decay_arguments_of_the_binding(dattn):
    with pytest.raises(ValueError):
        dattn._host_f32([0.0], 2, "log_decay")
    assert dattn._host_f32(None, 2, "log_decay") is None
