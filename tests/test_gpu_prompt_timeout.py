"""Waits of the prompt kernels that run out: the call ends with DATTN_ETIMEOUT, the states stay as they were, and the
next call is as if nothing had happened. As in test_gpu_timeout.py a testing aid withholds what is waited for - copies
that are not requested - and the limit is 200 us: nothing faults, traps or hangs."""
import time

import pytest
import torch

from test_gpu_linear import decays, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# (in one piece; cut into ranges; cut, three Q tiles a chunk and a stream that is whole; a head of its own)
CASES = [(4, 2, 128, [100]), (2, 1, 128, [1600]), (5, 1, 256, [1500, 70]), (1, 1, 256, [2000])]


@pytest.mark.parametrize("Hq,Hkv,D,count", CASES)
@pytest.mark.parametrize("what", ["q", "kv"])
def test_waits_that_run_out(dattn, Hq, Hkv, D, count, what):
    cut = max(count) > 1000
    g = torch.Generator().manual_seed(Hq + D)
    B, T = len(count), max(count)
    layer = {"kind": dattn.CACHE_STATE, "log_decay": decays(Hkv)}
    q, k, v, gate = (x.cuda() for x in inputs(g, B, T, Hq=Hq, Hkv=Hkv, D=D))
    start = torch.randn(B, Hkv, D, D, generator=g).cuda()
    n, zero = i32(count), i32([0] * B)

    def call(h, state):
        out = torch.full((B, T, Hq, D), 7.0, device="cuda")
        h.prefill(0, dattn.state_cache(state), q, k, v, n, zero, out, gate=gate)
        return out

    want_state = start.clone()
    fresh = dattn.Handle(Hq, Hkv, D, [layer], B)
    want = call(fresh, want_state)
    assert fresh.get_error() == dattn.OK

    h, state = dattn.Handle(Hq, Hkv, D, [layer], B), start.clone()
    h.debug_config(dattn.DEBUG_WITHHOLD_Q if what == "q" else dattn.DEBUG_WITHHOLD_KV, wait_limit_us=200)
    for _ in range(2):
        t0 = time.perf_counter()
        call(h, state)
        status = h.get_error()
        assert time.perf_counter() - t0 < 1.5, "the wait limit was not applied"
        if what == "kv" and not cut:  # (nothing is summed)
            assert status == dattn.OK
            state.copy_(start)
            continue
        assert status == dattn.ETIMEOUT
        assert h.get_error() == dattn.OK
        assert torch.equal(state, start)
    h.debug_config(0, 0)
    for _ in range(2):
        state.copy_(start)
        out = call(h, state)
        assert h.get_error() == dattn.OK
        assert torch.equal(out, want) and torch.equal(state, want_state)
