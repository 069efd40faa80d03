"""A stream whose length is outside the call's bound is reported and its cache left as it is: the new entry has no
slot that is known to be free (the clamped length names a live token of a longer stream)."""
import pytest
import torch

from test_gpu_sparse import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [16 * 45 + 1, 16 * 50, -3])
def test_sparse_decode_writes_nothing(dattn, fp8, bad):
    c = Case(41, 8, 2, 128, 16, [16 * 40 + 3, 16 * 50, 77], fp8=fp8)
    h = c.handle(dattn, 8, max_context=16 * 45)
    c.lens[1] = bad
    bits = lambda t: t.cpu().view(torch.uint8 if fp8 else torch.int16)  # noqa: E731
    k, v = bits(c.k).clone(), bits(c.v).clone()
    c.run(dattn, 8, 1, 1, write=True, handle=h, expect=dattn.ELENGTH)
    for b in (0, 2):
        n = c.lens[b]
        pg = int(c.table[b, n // 16])
        for j in range(2):
            k1, v1 = c.entries(b, j)
            k[pg, j, n % 16], v[pg, j, n % 16] = bits(k1), bits(v1)
    assert torch.equal(bits(c.kd), k) and torch.equal(bits(c.vd), v)
