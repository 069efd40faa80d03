"""Prompts on state layers that are cut into ranges: a CTA's range begins and ends
inside a stream, whose state the CTA before hands on. Tolerances as for the
prompt form (2^-16 + (D + 128) 2^-23 of the sum of the contributions' sizes, and
2^-24 a token for the state carried along)."""
import numpy as np
import pytest
import torch

from test_gpu_linear import Ref, close, decays, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def run(dattn, h, layer, state, q, k, v, gate, count, rows=None, out=None):
    B, T, Hq, D = q.shape
    out = torch.full((B, T, Hq, D), 7.0, device="cuda") if out is None else out
    d = lambda x: None if x is None else x.cuda()  # noqa: E731
    h.prefill(layer, dattn.state_cache(state, rows), d(q), d(k), d(v), i32(count), i32([0] * B), out, gate=d(gate))
    return out


@pytest.mark.parametrize("Hq,Hkv,D,count", [(5, 1, 256, [900]), (24, 4, 256, [641, 0, 65]), (8, 1, 128, [1500, 1, 64, 448]),
                                            (3, 1, 128, [1400]), (8, 8, 128, [700, 3]), (14, 2, 256, [70, 1000, 512])])
def test_layouts(dattn, Hq, Hkv, D, count):
    """Odd groups, groups of one and of eight, a gate; rows past a count hold NaN and are left alone."""
    g = torch.Generator().manual_seed(Hq * D + len(count))
    B, T = len(count), max(count) + 5
    ld = decays(Hkv)
    q, k, v, gate = inputs(g, B, T, Hq=Hq, Hkv=Hkv, D=D)
    for b, n in enumerate(count):
        for x in (q, k, v):
            x[b, n:] = float("nan")
    state = torch.randn(B + 1, Hkv, D, D, generator=g)
    rows = torch.arange(B, 0, -1, dtype=torch.int32)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], B)
    sd = state.cuda()
    out = run(dattn, h, 0, sd, q, k, v, gate, count, rows.cuda()).cpu()
    assert h.get_error() == dattn.OK
    ref = Ref(state, ld)
    eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23 + T * 2.0 ** -24
    for b, n in enumerate(count):
        for t in range(n):
            want, size = ref.step(int(rows[b]), q[b, t], k[b, t], v[b, t], gate[b, t])
            if t % 29 == 0 or t % 64 in (0, 63) or t > n - 3:
                close(out[b, t], want, size, eps, f"row {b} token {t}")
        assert (out[b, n:] == 7.0).all()
    close(sd.cpu(), ref.s, ref.a, eps, "state")
    assert torch.equal(sd.cpu()[0], state[0])


@pytest.mark.parametrize("D", [128, 256])
def test_missing_and_infinite_values_cross_the_ranges(dattn, D):
    """A value that is no number leaves its column's other tokens before it, and all other columns, as they are."""
    g = torch.Generator().manual_seed(D)
    Hq, Hkv, T, at, col = 2, 1, 1600, 777, 37
    ld = decays(Hkv)
    q, k, v, _ = inputs(g, 1, T, Hq=Hq, Hkv=Hkv, D=D)
    clean = v.clone()
    v[0, at, 0, col] = float("nan")
    v[0, at + 3, 0, col + 64] = float("inf")
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    s0, s1 = torch.zeros(1, Hkv, D, D, device="cuda"), torch.zeros(1, Hkv, D, D, device="cuda")
    a = run(dattn, h, 0, s0, q, k, clean, None, [T]).cpu()
    b = run(dattn, h, 0, s1, q, k, v, None, [T]).cpu()
    assert h.get_error() == dattn.OK
    other = [c for c in range(D) if c not in (col, col + 64)]
    assert torch.equal(a[..., other], b[..., other]) and torch.isfinite(a).all()
    assert torch.equal(s0.cpu()[..., other], s1.cpu()[..., other])
    for c, t in ((col, at), (col + 64, at + 3)):
        assert torch.equal(a[0, :t, :, c], b[0, :t, :, c])
        assert not torch.isfinite(b[0, t:, :, c]).any()


def test_bad_rows_and_counts_are_reported_and_left_alone(dattn):
    g = torch.Generator().manual_seed(4)
    Hq, Hkv, D, T = 4, 2, 128, 900
    ld = decays(Hkv)
    q, k, v, _ = inputs(g, 4, T, Hq=Hq, Hkv=Hkv, D=D)
    state = torch.randn(4, Hkv, D, D, generator=g)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 4)
    sd, rows, count = state.cuda(), [0, 9, 2, 3], [T, T, T + 1, T]
    out = run(dattn, h, 0, sd, q, k, v, None, count, i32(rows)).cpu()
    assert h.get_error() == dattn.EINDEX
    assert (out[1] == 7.0).all() and (out[2] == 7.0).all()
    assert torch.equal(sd.cpu()[1:3], state[1:3])
    want = state[[0, 3]].cuda()
    two = run(dattn, h, 0, want, q[[0, 3]], k[[0, 3]], v[[0, 3]], None, [T, T]).cpu()
    assert h.get_error() == dattn.OK
    ref = Ref(state, ld)
    eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23 + T * 2.0 ** -24
    for i, b in enumerate((0, 3)):
        for t in range(T):
            w, size = ref.step(b, q[b, t], k[b, t], v[b, t])
            if t % 97 == 0 or t == T - 1:
                close(out[b, t], w, size, eps, f"row {b} token {t}")
                close(two[i, t], w, size, eps, f"alone, row {b} token {t}")


def test_layers_share_the_workspace_in_a_graph(dattn):
    """Three prompts on two layers and a step behind them, captured once: the same bits as eager calls, every time."""
    g = torch.Generator().manual_seed(6)
    Hq, Hkv, D, T, B = 8, 2, 256, 1100, 2
    ld = decays(Hkv)
    layers = [{"kind": dattn.CACHE_STATE, "log_decay": ld}, {"kind": dattn.CACHE_STATE, "log_decay": ld * 3}]
    h = dattn.Handle(Hq, Hkv, D, layers, B)
    xs = [[x.cuda() for x in inputs(g, B, T, Hq=Hq, Hkv=Hkv, D=D)] for _ in range(3)]
    step = [x[:, 5].contiguous() for x in xs[0]]
    counts = [i32([T, 700]), i32([64, T]), i32([T, 1])]
    zero, pos = i32([0] * B), i32([T] * B)
    start = torch.randn(2, B, Hkv, D, D, generator=g).cuda()
    states = start.clone()
    caches = [dattn.state_cache(states[0]), dattn.state_cache(states[1])]
    outs = [torch.zeros(B, T, Hq, D, device="cuda") for _ in range(3)]
    last = torch.zeros(B, Hq, D, device="cuda")

    def calls():
        for i, layer in enumerate((0, 1, 0)):
            q, k, v, gate = xs[i]
            h.prefill(layer, caches[layer], q, k, v, counts[i], zero, outs[i], gate=gate)
        h.decode(0, caches[0], *step[:3], pos, last, gate=step[3])

    calls()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs + [last, states]]
    assert all(torch.isfinite(x).all() for x in want)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            calls()
        for _ in range(3):
            states.copy_(start)
            for x in outs + [last]:
                x.zero_()
            graph.replay()
            stream.synchronize()
            for x, y in zip(outs + [last, states], want):
                assert torch.equal(x, y)
    assert h.get_error(stream) == dattn.OK
