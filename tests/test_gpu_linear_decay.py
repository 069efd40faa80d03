"""A decay near 1 over many steps: what fp32 drops of it counts."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_decays_between_two_floats():
    """Decays whose fp32 rounding is off by 2.98e-8 (as far as it can be) in either direction, over 3,000 steps: 9e-5 of
    the state if that were dropped. A step rounds each element once, by 2^-24 / sqrt(3) at most in root mean square:
    six times that over 3,000 steps for the worst of 32,768 elements, 1.1e-5."""
    import decode_attention_kv_dattn_gb300 as dattn
    ld = np.array([-(2.0 ** -12), -float.fromhex("0x1.001p-12")], np.float32)
    lam = np.exp(ld.astype(np.float64))
    lost = lam - lam.astype(np.float32)
    assert abs(lost[0] - 2.98e-8) < 1e-10 and abs(lost[1] + 2.98e-8) < 1e-10
    Hq, Hkv, D, n = 2, 2, 128, 3000
    g = torch.Generator().manual_seed(3)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    start = torch.randn(1, Hkv, D, D, generator=g)
    sd = start.cuda()
    cache, pos = dattn.state_cache(sd), torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(1, Hq, D, generator=g).to(torch.bfloat16).cuda()
    zero = torch.zeros(1, Hkv, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(1, Hq, D, device="cuda")
    for _ in range(n):
        h.decode(0, cache, q, zero, zero, pos, out)
    assert h.get_error() == dattn.OK
    want = start.double() * torch.from_numpy(np.exp(ld.astype(np.float64) * n)).view(1, Hkv, 1, 1)
    off = (sd.cpu().double() / want - 1).abs().max().item()
    assert off <= 6 * math.sqrt(n) * 2.0 ** -24 / math.sqrt(3)
