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


def dense(dattn, c, max_context, **kw):
    """dattn_decode with write-back on the case's stream lengths: status, K and V pools."""
    B = len(c.lens)
    h = dattn.Handle(c.Hq, c.Hkv, c.D, [c.layer(dattn)], B, max_context=max_context)
    kd, vd = c.k.cuda(), c.v.cuda()
    cache = dattn.paged_cache(kd, vd, c.table.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda())
    out = torch.empty(B, c.Hq, c.D, device="cuda")
    args = (0, cache, c.q.cuda(), c.k_new.cuda(), c.v_new.cuda(), c.pos.cuda(), out)
    if kw.pop("noalloc", False):
        dattn.decode_noalloc(h.config, *args, **kw)
        torch.cuda.synchronize()
        status = dattn.ELENGTH
    else:
        h.decode(*args, **kw)
        status = h.get_error()
    return status, kd, vd


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [16 * 45 + 1, 16 * 50, 16 * 51, -3])
def test_decode_writes_nothing(dattn, fp8, bad):
    """The bound of max_seq_len, and the table's end."""
    c = Case(42, 8, 2, 128, 16, [16 * 40 + 3, 16 * 50, 77], fp8=fp8)
    c.lens[1] = bad
    bits = lambda t: t.cpu().view(torch.uint8 if fp8 else torch.int16)  # noqa: E731
    k, v = bits(c.k).clone(), bits(c.v).clone()
    for b in (0, 2):
        n = c.lens[b]
        pg = int(c.table[b, n // 16])
        for j in range(2):
            k1, v1 = c.entries(b, j)
            k[pg, j, n % 16], v[pg, j, n % 16] = bits(k1), bits(v1)
    for noalloc in ([False] if fp8 else [False, True]):
        status, kd, vd = dense(dattn, c, 16 * 60, max_seq_len=16 * 45, noalloc=noalloc)
        assert status == dattn.ELENGTH
        assert torch.equal(bits(kd), k) and torch.equal(bits(vd), v)


@pytest.mark.parametrize("bad", [16 * 45 + 1, 16 * 50, -3])
def test_verify_writes_nothing(dattn, bad):
    """The other streams' windows land behind their prefixes."""
    T = 5
    c = Case(43, 8, 2, 256, 16, [16 * 40 + 3, 16 * 50 + T, 77 + T])
    c.lens = [16 * 40 + 3, bad, 77]
    x = lambda *s: torch.randn(*s, generator=c.g).to(torch.bfloat16)  # noqa: E731
    q, k, v = x(3, T, 8, 256), x(3, T, 2, 256), x(3, T, 2, 256)
    h = dattn.Handle(8, 2, 256, [c.layer(dattn)], 3, max_context=16 * 60, max_verify_rows=T)
    kd, vd = c.k.cuda(), c.v.cuda()
    nd = torch.tensor(c.lens, dtype=torch.int32).cuda()
    parent = (torch.arange(T, dtype=torch.int32) - 1).repeat(3, 1).cuda()
    out = torch.empty(3, T, 8, 256, device="cuda")
    h.verify(0, dattn.paged_cache(kd, vd, c.table.cuda(), nd), q.cuda(), k.cuda(), v.cuda(), parent, out,
             max_prefix_len=16 * 45, pos=torch.zeros(3, dtype=torch.int32).cuda())
    assert h.get_error() == dattn.ELENGTH
    want = c.v.clone()
    for b in (0, 2):
        for i in range(T):
            n = c.lens[b] + i
            want[int(c.table[b, n // 16]), :, n % 16] = v[b, i]
    assert torch.equal(vd.cpu(), want)
    pages = [int(p) for p in c.table[1] if p >= 0]
    assert torch.equal(kd.cpu()[pages], c.k[pages])
