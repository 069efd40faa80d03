"""Linear attention with a decay for each head on the GPU: the step (decode on
a state layer) and the prompt form (prefill) against the recurrence in 64 bits.

Tolerances, per element, relative to the same recurrence over absolute values
(the sum of all contributions' sizes): the step's sums are fp32, D products and
the decay - (D + 8) 2^-24. The prompt form adds what two bf16 terms drop of a
32-bit operand (2^-17 for each of two in a product) and sums in chunks:
2^-16 + (D + 128) 2^-23; a state carried over `n` tokens is rounded once a
chunk or token, so n 2^-24 more at most.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def sigmoid(x):
    return 1 / (1 + torch.exp(-x.double()))


class Ref:
    """The recurrence over float64 states, and over absolute values beside it."""

    def __init__(self, state, log_decay):
        self.s, self.a = state.double(), state.double().abs()
        self.lam = torch.exp(torch.as_tensor(log_decay, dtype=torch.float32).double()).view(-1, 1, 1)

    def step(self, b, q, k, v, gate=None, keep=True):
        """One token of row b: q [Hq, D], k, v [Hkv, D]; returns (out, size) [Hq, D]."""
        kv = k.double()[:, :, None] * v.double()[:, None]
        s, a = self.s[b] * self.lam + kv, self.a[b] * self.lam + kv.abs()
        if keep:
            self.s[b], self.a[b] = s, a
        G, D = q.shape[0] // k.shape[0], q.shape[1]
        f = 1 / math.sqrt(D)
        out = torch.einsum("hgd,hde->hge", q.double().view(-1, G, D), s).reshape(-1, D) * f
        size = torch.einsum("hgd,hde->hge", q.double().abs().view(-1, G, D), a).reshape(-1, D) * f
        if gate is not None:
            out, size = out * sigmoid(gate)[:, None], size * sigmoid(gate)[:, None]
        return out, size


def decays(H):
    return np.log1p(-np.exp2(-5.0 - np.arange(H))).astype(np.float32)


def inputs(g, *lead, Hq, Hkv, D):
    rn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    return rn(*lead, Hq, D), rn(*lead, Hkv, D), rn(*lead, Hkv, D), rn(*lead, Hq)


def close(got, want, size, eps, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    d = (got - want).abs() - eps * size
    assert (d <= 0).all(), f"{what}: {d.max():.3g} over the bound, at a size of {size.flatten()[d.argmax()]:.3g}"


LAYOUTS = [(8, 2, 256), (16, 8, 128), (24, 4, 256), (4, 4, 128), (5, 1, 256), (6, 2, 128), (8, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", LAYOUTS)
@pytest.mark.parametrize("B", [1, 3])
def test_step(dattn, Hq, Hkv, D, B):
    g = torch.Generator().manual_seed(Hq + D + B)
    rows = torch.tensor([4, 0, 2][:B], dtype=torch.int32)
    state = torch.randn(5, Hkv, D, D, generator=g)
    ld = decays(Hkv)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], B)
    ref, sd = Ref(state, ld), state.cuda()
    cache = dattn.state_cache(sd, rows.cuda())
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    eps = (D + 8) * 2.0 ** -24
    for i in range(4):
        q, k, v, gate = inputs(g, B, Hq=Hq, Hkv=Hkv, D=D)
        gate = gate if i % 2 else None
        write = i != 1
        out = torch.full((B, Hq, D), float("nan"), device="cuda")
        h.decode(0, cache, q.cuda(), k.cuda(), v.cuda(), pos, out, gate=None if gate is None else gate.cuda(),
                 write_back=write)
        assert h.get_error() == dattn.OK
        for b in range(B):
            want, size = ref.step(int(rows[b]), q[b], k[b], v[b], None if gate is None else gate[b], keep=write)
            close(out[b].cpu(), want, size, eps + i * 2.0 ** -23, f"step {i} row {b}")
        close(sd.cpu(), ref.s, ref.a, (i + 2) * 2.0 ** -23, f"state {i}")
    untouched = [r for r in range(5) if r not in rows.tolist()]
    assert torch.equal(sd.cpu()[untouched], state[untouched])


def test_slow_decay_over_many_steps(dattn):
    """A decay of 1 - 2^-12 over 3,000 steps: what fp32 drops of it (2^-25 a step) would show as 2^-13.5."""
    g = torch.Generator().manual_seed(3)
    Hq, Hkv, D = 2, 2, 128
    ld = np.log1p(-np.exp2(-np.array([12.0, 13.0]))).astype(np.float32)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    sd = torch.ones(1, Hkv, D, D, device="cuda")
    cache, pos = dattn.state_cache(sd), torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(1, Hq, D, generator=g).to(torch.bfloat16).cuda()
    zero = torch.zeros(1, Hkv, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(1, Hq, D, device="cuda")
    n = 3000
    for _ in range(n):
        h.decode(0, cache, q, zero, zero, pos, out)
    assert h.get_error() == dattn.OK
    want = torch.exp(torch.from_numpy(ld).double() * n).view(1, Hkv, 1, 1).expand(1, Hkv, D, D)
    # each step rounds the state once: a random walk of 3,000 half steps of 2^-24, with room for twice that
    assert ((sd.cpu().double() / want - 1).abs() <= 2 * math.sqrt(n) * 2.0 ** -24 * 4).all()


@pytest.mark.parametrize("Hq,Hkv,D", LAYOUTS)
@pytest.mark.parametrize("T,count", [(1, [1, 0]), (64, [64, 63]), (65, [65, 1]), (200, [129, 200]), (17, [0, 17])])
def test_prompt(dattn, Hq, Hkv, D, T, count):
    g = torch.Generator().manual_seed(Hq + D + T)
    B = len(count)
    rows = torch.tensor([2, 0], dtype=torch.int32)
    state = torch.randn(3, Hkv, D, D, generator=g)
    ld = decays(Hkv)
    q, k, v, gate = inputs(g, B, T, Hq=Hq, Hkv=Hkv, D=D)
    gate = gate if T % 2 else None
    # rows past a count are not read
    for b in range(B):
        for x in (q, k, v):
            x[b, count[b]:] = float("nan")
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], B)
    sd = state.cuda()
    out = torch.full((B, T, Hq, D), 7.0, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    h.prefill(0, dattn.state_cache(sd, rows.cuda()), q.cuda(), k.cuda(), v.cuda(), i32(count), i32([0] * B), out,
              gate=None if gate is None else gate.cuda())
    assert h.get_error() == dattn.OK
    ref, out = Ref(state, ld), out.cpu()
    eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23
    for b in range(B):
        for t in range(count[b]):
            want, size = ref.step(int(rows[b]), q[b, t], k[b, t], v[b, t], None if gate is None else gate[b, t])
            close(out[b, t], want, size, eps, f"row {b} token {t}")
        assert (out[b, count[b]:] == 7.0).all()
    close(sd.cpu(), ref.s, ref.a, eps, "state")
    assert torch.equal(sd.cpu()[1], state[1])
    for b in range(B):
        if count[b] == 0:
            assert torch.equal(sd.cpu()[rows[b]], state[rows[b]])


@pytest.mark.parametrize("Hq,Hkv,D,T,B", [(4, 2, 128, 2500, 1), (8, 2, 256, 1100, 1), (4, 4, 128, 700, 5)])
def test_long_prompt(dattn, Hq, Hkv, D, T, B):
    """Long enough to be cut into segments; decays from none at all to one that is gone after a token."""
    g = torch.Generator().manual_seed(T)
    ld = np.array([0.0, -20.0, -1e-4, -200.0][:Hkv], np.float32)
    state = torch.randn(B, Hkv, D, D, generator=g)
    q, k, v, _ = inputs(g, B, T, Hq=Hq, Hkv=Hkv, D=D)
    count = [T - 7 * b for b in range(B)]
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], B)
    sd = state.cuda()
    out = torch.full((B, T, Hq, D), 7.0, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    h.prefill(0, dattn.state_cache(sd), q.cuda(), k.cuda(), v.cuda(), i32(count), i32([0] * B), out)
    assert h.get_error() == dattn.OK
    ref, out = Ref(state, ld), out.cpu()
    eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23 + T * 2.0 ** -24
    for b in range(B):
        for t in range(count[b]):
            want, size = ref.step(b, q[b, t], k[b, t], v[b, t])
            if t % 37 == 0 or t > count[b] - 3:
                close(out[b, t], want, size, eps, f"row {b} token {t}")
        assert (out[b, count[b]:] == 7.0).all()
    close(sd.cpu(), ref.s, ref.a, eps, "state")


def test_prompt_in_pieces_then_steps(dattn):
    """A prompt in two calls, then steps: the same as one call over all tokens, within both sides' bounds."""
    g = torch.Generator().manual_seed(9)
    Hq, Hkv, D, T = 6, 2, 128, 150
    ld = decays(Hkv)
    q, k, v, gate = inputs(g, 1, T, Hq=Hq, Hkv=Hkv, D=D)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    sd = torch.zeros(1, Hkv, D, D, device="cuda")
    cache = dattn.state_cache(sd)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    out = torch.empty(1, T, Hq, D, device="cuda")
    for lo, hi in ((0, 70), (70, 141)):
        part = [x[:, lo:hi].contiguous().cuda() for x in (q, k, v, gate)]
        o = torch.empty(1, hi - lo, Hq, D, device="cuda")
        h.prefill(0, cache, *part[:3], i32([hi - lo]), i32([lo]), o, gate=part[3])
        out[:, lo:hi] = o
    for t in range(141, T):
        o = torch.empty(1, Hq, D, device="cuda")
        h.decode(0, cache, *(x[:, t].contiguous().cuda() for x in (q, k, v)), i32([t]), o, gate=gate[:, t].contiguous().cuda())
        out[:, t] = o
    assert h.get_error() == dattn.OK
    ref = Ref(torch.zeros(1, Hkv, D, D), ld)
    eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23
    for t in range(T):
        want, size = ref.step(0, q[0, t], k[0, t], v[0, t], gate[0, t])
        close(out[0, t].cpu(), want, size, eps, f"token {t}")


def test_infinite_and_missing_values_stay_with_their_stream(dattn):
    """An infinity in one row's state or keys does not reach the others."""
    g = torch.Generator().manual_seed(4)
    Hq, Hkv, D, T = 4, 2, 128, 70
    q, k, v, _ = inputs(g, 2, T, Hq=Hq, Hkv=Hkv, D=D)
    k[0, 3, 0, 5] = float("inf")
    ld = decays(Hkv)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 2)
    sd = torch.zeros(2, Hkv, D, D, device="cuda")
    out = torch.zeros(2, T, Hq, D, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    h.prefill(0, dattn.state_cache(sd), q.cuda(), k.cuda(), v.cuda(), i32([T, T]), i32([0, 0]), out)
    assert h.get_error() == dattn.OK
    assert torch.isfinite(out[1]).all() and torch.isfinite(sd[1]).all()
    assert torch.isfinite(out[0, :3]).all() and not torch.isfinite(out[0, 3:, :2]).any()
    assert torch.isfinite(out[0, :, 2:]).all()


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 2), (256, 3, 1)])
def test_values_that_are_no_numbers_reach_no_earlier_token(dattn, D, Hq, Hkv):
    """An infinity in v: its column has no number from its token on, everything before it and every other column
    is as without it. A NaN in q: its own row."""
    g = torch.Generator().manual_seed(14)
    T, at, e = 150, 75, D - 3
    ld = decays(Hkv)
    q, k, v, _ = inputs(g, 1, T, Hq=Hq, Hkv=Hkv, D=D)
    bad = v.clone()
    bad[0, at, 0, e] = float("inf")
    bad[0, at + 20, 0, e] = float("nan")
    bq = q.clone()
    bq[0, at - 5, 0, 1] = float("nan")
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    runs = []
    for qq, vv in ((q, v), (bq, bad)):
        sd, out = torch.zeros(1, Hkv, D, D, device="cuda"), torch.zeros(1, T, Hq, D, device="cuda")
        h.prefill(0, dattn.state_cache(sd), qq.cuda(), k.cuda(), vv.cuda(), i32([T]), i32([0]), out)
        assert h.get_error() == dattn.OK
        runs.append((out.cpu()[0], sd.cpu()[0]))
    (o0, s0), (o1, s1) = runs
    G = Hq // Hkv
    clean = torch.ones_like(o0, dtype=torch.bool)
    clean[at:, :G, e] = False
    clean[at - 5, 0] = False
    assert torch.equal(o0[clean], o1[clean])
    assert not torch.isfinite(o1[~clean]).any()
    keep = torch.ones_like(s0, dtype=torch.bool)
    keep[0, :, e] = False
    assert torch.equal(s0[keep], s1[keep]) and not torch.isfinite(s1[0, :, e]).any()


@pytest.mark.parametrize("count", [[1000, 3, 0, 700, 64], [0, 0, 0, 0, 1], [0] * 5, [320, 320, 320, 320, 320]])
def test_ragged_batch_cut_into_ranges(dattn, count):
    """Streams of very different lengths, none at all, and lengths whose ranges end on unit borders."""
    g = torch.Generator().manual_seed(15)
    Hq, Hkv, D, B = 6, 3, 128, len(count)
    T = max(max(count), 400)
    ld = np.array([0.0, -0.003, -0.2], np.float32)
    state = torch.randn(B, Hkv, D, D, generator=g)
    q, k, v, _ = inputs(g, B, T, Hq=Hq, Hkv=Hkv, D=D)
    for b in range(B):
        for x in (q, k, v):
            x[b, count[b]:] = float("nan")
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], B)
    sd, out = state.cuda(), torch.full((B, T, Hq, D), 7.0, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    h.prefill(0, dattn.state_cache(sd), q.cuda(), k.cuda(), v.cuda(), i32(count), i32([0] * B), out)
    assert h.get_error() == dattn.OK
    ref, out = Ref(state, ld), out.cpu()
    eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23 + T * 2.0 ** -24
    for b in range(B):
        for t in range(count[b]):
            want, size = ref.step(b, q[b, t], k[b, t], v[b, t])
            if t % 29 == 0 or t > count[b] - 3:
                close(out[b, t], want, size, eps, f"row {b} token {t}")
        assert (out[b, count[b]:] == 7.0).all()
        if count[b] == 0:
            assert torch.equal(sd[b].cpu(), state[b])
    close(sd.cpu(), ref.s, ref.a, eps, "state")


def test_outputs_and_states_on_16_byte_boundaries(dattn):
    g = torch.Generator().manual_seed(8)
    Hq, Hkv, D, T = 4, 2, 128, 66
    ld = decays(Hkv)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    q, k, v, _ = inputs(g, 1, T, Hq=Hq, Hkv=Hkv, D=D)
    shifted = lambda *s: torch.zeros(math.prod(s) + 8, device="cuda")[4:-4].view(*s)  # noqa: E731
    sd, out = shifted(1, Hkv, D, D), shifted(1, T, Hq, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    h.prefill(0, dattn.state_cache(sd), q.cuda(), k.cuda(), v.cuda(), i32([T]), i32([0]), out)
    assert h.get_error() == dattn.OK
    ref = Ref(torch.zeros(1, Hkv, D, D), ld)
    for t in range(T):
        want, size = ref.step(0, q[0, t], k[0, t], v[0, t])
        close(out[0, t].cpu(), want, size, 2.0 ** -16 + (D + 128) * 2.0 ** -23, f"token {t}")
    close(sd.cpu(), ref.s, ref.a, 2.0 ** -16 + (D + 128) * 2.0 ** -23, "state")


def test_bad_metadata_is_reported(dattn):
    Hq, Hkv, D, T = 4, 2, 128, 8
    g = torch.Generator().manual_seed(5)
    q, k, v, _ = (x.cuda() for x in inputs(g, 2, T, Hq=Hq, Hkv=Hkv, D=D))
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": decays(Hkv)}], 2)
    state = torch.randn(2, Hkv, D, D, generator=g)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for rows, count in (([0, 2], [T, T]), ([-1, 1], [T, T]), ([0, 1], [T + 1, T]), ([0, 1], [T, -1])):
        sd = state.cuda()
        out = torch.full((2, T, Hq, D), 7.0, device="cuda")
        h.prefill(0, dattn.state_cache(sd, i32(rows)), q, k, v, i32(count), i32([0, 0]), out)
        assert h.get_error() == dattn.EINDEX
        for b in range(2):
            ok = 0 <= rows[b] < 2 and 0 <= count[b] <= T
            assert bool((out[b] == 7.0).all()) != ok
            if not ok and 0 <= rows[b] < 2:
                assert torch.equal(sd[rows[b]].cpu(), state[rows[b]])
    sd = state.cuda()
    out = torch.full((2, Hq, D), 7.0, device="cuda")
    h.decode(0, dattn.state_cache(sd, i32([0, 9])), q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
             i32([0, 0]), out)
    assert h.get_error() == dattn.EINDEX
    assert torch.equal(sd[1].cpu(), state[1]) and not torch.equal(sd[0].cpu(), state[0])


def test_refusals(dattn):
    state = {"kind": dattn.CACHE_STATE, "log_decay": np.zeros(2, np.float32)}

    def refused(code, call):
        with pytest.raises(dattn.DattnError) as e:
            call()
        assert e.value.code == code

    h = dattn.Handle(4, 2, 128, [state], 2, max_verify_rows=4)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    sd = torch.zeros(3, 2, 128, 128, device="cuda")
    cache, n = dattn.state_cache(sd), i32([0, 0, 0])
    out = torch.zeros(3, 4, 128, device="cuda")
    refused(dattn.EXCEEDS, lambda: h.decode(0, cache, bf(3, 4, 128), bf(3, 2, 128), bf(3, 2, 128), n, out))
    refused(dattn.EXCEEDS, lambda: h.prefill(0, cache, bf(3, 1, 4, 128), bf(3, 1, 2, 128), bf(3, 1, 2, 128), n, n, out))
    refused(dattn.EUNSUPPORTED, lambda: h.append_kv(0, cache, bf(1, 1, 2, 128), bf(1, 1, 2, 128), n, n, n))
    refused(dattn.EUNSUPPORTED, lambda: h.verify(0, cache, bf(1, 1, 4, 128), bf(1, 1, 2, 128), bf(1, 1, 2, 128),
                                                 i32([[-1]]), out, write_back=False))
    refused(dattn.EUNSUPPORTED, lambda: h.commit(0, cache, bf(1, 1, 2, 128), bf(1, 1, 2, 128), i32([[-1]]), i32([[0]]), n, n))
    refused(dattn.EUNSUPPORTED, lambda: dattn.decode_noalloc(h.config, 0, cache, bf(1, 4, 128), bf(1, 2, 128),
                                                             bf(1, 2, 128), n, out))
    refused(dattn.EUNSUPPORTED, lambda: h.sparse_decode(0, cache, bf(1, 2, 128), bf(1, 4, 128), bf(1, 2, 128),
                                                        bf(1, 2, 128), n, out, 1, keep_first=0))
    assert h.get_error() == dattn.OK


def test_graph_replay_on_a_side_stream(dattn):
    """A captured prompt and step, replayed: the state moves on with each replay."""
    g = torch.Generator().manual_seed(6)
    Hq, Hkv, D, T = 8, 2, 256, 100
    ld = decays(Hkv)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    q, k, v, gate = inputs(g, 1, T, Hq=Hq, Hkv=Hkv, D=D)
    d = [x.cuda() for x in (q, k, v, gate)]
    one = [x[:, 0].contiguous() for x in d]
    sd = torch.zeros(1, Hkv, D, D, device="cuda")
    cache = dattn.state_cache(sd)
    n, pos = torch.tensor([T], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    out, o1 = torch.empty(1, T, Hq, D, device="cuda"), torch.empty(1, Hq, D, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            h.prefill(0, cache, *d[:3], n, pos, out, gate=d[3])
            h.decode(0, cache, *one[:3], pos, o1, gate=one[3])
        sd.zero_()
        for _ in range(2):
            graph.replay()
        stream.synchronize()
    assert h.get_error() == dattn.OK
    ref = Ref(torch.zeros(1, Hkv, D, D), ld)
    for _ in range(2):
        for t in range(T):
            want, size = ref.step(0, q[0, t], k[0, t], v[0, t], gate[0, t])
        last, ls = ref.step(0, q[0, 0], k[0, 0], v[0, 0], gate[0, 0])
    eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23
    close(out[0, T - 1].cpu(), want, size, eps)
    close(o1[0].cpu(), last, ls, eps)
    close(sd.cpu(), ref.s, ref.a, eps)
