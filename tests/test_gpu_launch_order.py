"""The order in which a captured run of calls is launched: behind a read-back, whose rows
may be the next call's inputs, a kernel waits for the whole of it, unless it reads no
inputs before it waits (append, read-back, a 4-bit layer's decode); behind a decode it may
start while that ends. Read from the graph's edges; nothing is launched."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def edge_types(graph):
    """Types of the edges of a chain of kernels, first to last (0: full order, 1: programmatic)."""
    cuda = ctypes.CDLL("libcuda.so.1")
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cuda.cuGraphGetEdges_v2(raw, None, None, None, ctypes.byref(n)) == 0
    src, dst, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (ctypes.c_uint8 * (8 * n.value))()
    assert cuda.cuGraphGetEdges_v2(raw, src, dst, data, ctypes.byref(n)) == 0
    nxt = {src[i]: (dst[i], data[8 * i + 2]) for i in range(n.value)}
    assert len(nxt) == n.value  # a chain
    at, types = (set(src) - set(dst)).pop(), []
    while at in nxt:
        at, t = nxt[at]
        types.append(t)
    return types


@pytest.mark.parametrize("fmt", ["KV_BF16", "KV_E4M3", "KV_INT4"])
def test_what_follows_a_read_back_waits_for_all_of_it(fmt):
    import decode_attention_kv_dattn_gb300 as dattn
    B, H, D, P, pages = 2, 2, 128, 16, 8
    h = dattn.Handle(8, H, D, [{"kind": dattn.CACHE_PAGED, "page_size": P, "kv_format": f, "k_scale": 1.0, "v_scale": 1.0}
                               for f in (getattr(dattn, fmt), dattn.KV_INT4, dattn.KV_BF16)], B, max_context=64,
                     max_verify_rows=4)

    def cache(fmt):
        if fmt == "KV_INT4":
            pools = [dattn.int4_pool(pages, H, P, D) for _ in range(2)]
        else:
            pools = [torch.zeros(pages, H, P, D, dtype=torch.uint8 if fmt == "KV_E4M3" else torch.bfloat16, device="cuda")
                     for _ in range(2)]
        return dattn.paged_cache(*pools, torch.arange(pages, dtype=torch.int32, device="cuda").view(B, -1),
                                 torch.full((B,), 5, dtype=torch.int32, device="cuda"))

    caches = [cache(fmt), cache("KV_INT4"), cache("KV_BF16")]
    x = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    z, one = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    q, k, v, out = x(B, 8, D), x(B, 1, H, D), x(B, 1, H, D), torch.zeros(B, 8, D, device="cuda")
    kk, qq, wide, parent = x(B, 2, H, D), x(B, 2, 8, D), torch.zeros(B, 2, 8, D, device="cuda"), torch.tensor(
        [[-1, 0]] * B, dtype=torch.int32, device="cuda")
    read = lambda: h.read_kv(0, caches[0], z, one, k, v)  # noqa: E731
    decode = lambda i: h.decode(i, caches[i], q, k[:, 0], v[:, 0], one, out, write_back=False)  # noqa: E731
    append = lambda i: h.append_kv(i, caches[i], k, v, z, one, rotate=False)  # noqa: E731
    verify = lambda i: h.verify(i, caches[i], qq, kk, kk, parent, wide, write_back=False)  # noqa: E731
    runs = [
        (lambda: (decode(1), read(), decode(1), decode(2), read(), decode(2), read(), append(1), decode(2)), [1, 1, 1, 1, 0, 1, 1, 1]),
        (lambda: (read(), read(), verify(2)), [1, 0, 1, 1]),
    ]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for run, want in runs:
        g = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(g, stream=side):
            run()
        assert edge_types(g) == want
