"""How near decode over 4-bit caches is to 64-bit arithmetic over the same entries: the
root mean square of the outputs' errors against that of the outputs, on contexts of up
to 300,000 tokens.

The bound. Keys, values and queries are normal numbers around zero, so outputs shrink with
the context like their errors do, and an error of one weight's size relative to the weight
is one of the output's. A score's parts s (q_G . c_G) and b sum(q_G) are about 1.3 each, after
1 / sqrt(D), for each of the D / 64 groups; four MMA sums cut off within 2^-23 (0.58 of it on
average) and two roundings of 2^-24 in each leave 3 x 2^-23 over four groups, 3.6e-7. q's and the
weights' two fp16 terms add 2^-24 of a product each (they are off by 2^-22 at the most), the
outputs' fp32 sums of the few hundred keys of a warp less than that: 5e-7 in all, and 1e-6 is
twice that. What the kernel does against larger errors is then seen. With one of these gone the
error is above it: MMA sums of two blocks (3e-6 to 6e-6 at 300,001 tokens in one chain), centred
codes (3e-6 at 4,401 tokens, 2e-5 at 300,001), the weights' second term (2e-4), normal operands
of the keys (2e-6).
"""
import numpy as np
import pytest
import torch

import int4_ref as ref
from gpu_util import dev

pytestmark = pytest.mark.gpu
BOUND = 1e-6


def values(pool, side, D, n):
    """The first n tokens of a pool whose pages lie in order, one KV head: fp64 [n, D] on the device."""
    blocks = pool.view(-1, 9 * D)[:(n + 15) // 16]
    r, d = np.arange(16)[:, None], np.arange(D)[None]
    at = dev(np.asarray(ref.code_byte(side, D, r, d), np.int64)).view(-1)
    code = (blocks[:, at].view(-1, 16, D) >> dev((d % 2 * 4).astype(np.uint8))) & 15
    pairs = blocks[:, 8 * D:].contiguous().view(torch.bfloat16).view(-1, 16, D // 64, 2).double()
    x = pairs[..., :1] + code.view(-1, 16, D // 64, 64).double() * pairs[..., 1:]
    return x.view(-1, D)[:n]


@pytest.mark.parametrize("G,D", [(4, 256), (6, 256), (2, 128), (8, 128)])
@pytest.mark.parametrize("lens", [[300001], [40000, 33, 3000, 17777], [1 + 400 * i for i in range(12)]])
def test_error_against_64_bits(G, D, lens):
    import decode_attention_kv_dattn_gb300 as dattn
    B, P = len(lens), 64
    gen = torch.Generator("cuda").manual_seed(1000 * G + D + B)
    h = dattn.Handle(G, 1, D, [{"kind": dattn.CACHE_PAGED, "page_size": P, "kv_format": dattn.KV_INT4}], B,
                     max_context=max(lens))
    q, kn, vn = (torch.randn(B, x, D, generator=gen, device="cuda").bfloat16() for x in (G, 1, 1))
    out, seq = torch.zeros(B, G, D, device="cuda"), dev(np.array(lens, np.int32))
    room = [n // P + 1 for n in lens]
    first = np.cumsum([0] + room)
    bt = np.full((B, max(room)), -1, np.int32)
    for b in range(B):
        bt[b, :room[b]] = first[b] + np.arange(room[b])
    pools = [dattn.int4_pool(int(first[-1]), 1, P, D) for _ in range(2)]
    cache, step = dattn.paged_cache(*pools, dev(bt), seq), 60000
    for t in range(0, max(lens), step):
        n = min(step, max(lens) - t)
        k, v = (torch.randn(B, n, 1, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
        h.append_kv(0, cache, k, v, torch.full_like(seq, t), (seq - t).clamp(0, n), rotate=False)
    h.decode(0, cache, q, kn, vn, seq, out)  # (the new entry is written behind the others)
    assert h.get_error() == dattn.OK
    worst = 0.0  # of the streams, whose outputs differ in size
    for b, n in enumerate(lens):
        k, v = (values(p[first[b]:first[b + 1]], s, D, n + 1) for s, p in zip("kv", pools))
        a = torch.softmax(q[b].double() @ k.T / D ** 0.5, -1)
        want = a @ v
        worst = max(worst, float(((out[b].double() - want) ** 2).mean() ** 0.5 / (want ** 2).mean() ** 0.5))
    assert worst <= BOUND, f"{worst:.3g} of the outputs' size"
