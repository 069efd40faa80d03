"""An append of more rows than a grid has is refused before a launch is tried."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["KV_BF16", "KV_INT4"])
def test_rows_past_the_grid(fmt):
    import decode_attention_kv_dattn_gb300 as dattn
    H, D, P, B = 1, 128, 16, 65536
    h = dattn.Handle(H, H, D, [{"kind": dattn.CACHE_PAGED, "page_size": P, "kv_format": getattr(dattn, fmt)}], 1, max_context=16)
    pools = [dattn.int4_pool(1, H, P, D) if fmt == "KV_INT4" else torch.zeros(1, H, P, D, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache = dattn.paged_cache(*pools, zero.view(B, 1), zero)
    x = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dattn.DattnError) as e:
        h.append_kv(0, cache, x, x, zero, zero, rotate=False)
    assert e.value.code == dattn.EXCEEDS
    with pytest.raises(dattn.DattnError) as e:
        h.read_kv(0, cache, zero, zero, x, x)
    assert e.value.code == dattn.EXCEEDS
    # the most there may be, none of which brings a token
    h.append_kv(0, cache, x[1:], x[1:], zero[1:], zero[1:], rotate=False)
    assert h.get_error() == dattn.OK
