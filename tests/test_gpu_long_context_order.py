"""Calls of different kinds behind one another on a handle, without a wait in between, and two handles on two streams:
the bits are those of each call on its own."""
import pytest
import torch

from test_gpu_linear import decays, inputs
from test_gpu_sparse import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Mixed:
    """A handle with two paged layers (pages of 16 and of 24 tokens, so different selections) and a state layer."""

    def __init__(self, dattn, seed, num=9):
        self.dattn, self.num = dattn, num
        self.cases = [Case(seed, 8, 2, 256, P, [40 * P + 3, 7, 0, 25 * P], r=64) for P in (16, 24)]
        layers = [c.layer(dattn) for c in self.cases] + [{"kind": dattn.CACHE_STATE, "log_decay": decays(2)}]
        self.h = dattn.Handle(8, 2, 256, layers, 4, max_context=40 * 24 + 3, max_selected_pages=num)
        self.pools = [(c.k.cuda(), c.v.cuda(), c.summary.cuda(), c.table.cuda(), i32(c.lens)) for c in self.cases]
        self.caches = [dattn.paged_cache(k, v, t, n) for k, v, _, t, n in self.pools]
        g = torch.Generator().manual_seed(seed)
        self.prompt = [x.cuda() for x in inputs(g, 4, 500, Hq=8, Hkv=2, D=256)]
        self.counts, self.zero = i32([500, 3, 0, 450]), i32([0] * 4)
        self.start = torch.randn(4, 2, 256, 256, generator=g).cuda()
        self.steps = [[x.cuda() for x in inputs(g, 4, Hq=8, Hkv=2, D=256)] for _ in range(6)]
        self.pos = i32([5, 6, 7, 8])

    def new(self):
        return torch.full((4, 8, 256), float("nan"), device="cuda")

    def calls(self, wait):
        """Every kind of call, some twice in a row; the outputs."""
        state = self.start.clone()
        cache = self.dattn.state_cache(state)
        outs = []

        def done(*x):
            outs.extend(x)
            if wait:
                torch.cuda.current_stream().synchronize()

        for i in (0, 1, 2, 3, 4, 5):
            q, k, v, gate = self.steps[i]
            layer = i % 2
            for kind in ("sd", "ds", "ss", "dd", "sx", "xs")[i]:
                o = self.new()
                if kind == "s":
                    sel = torch.full((4, 2, self.num), -7, dtype=torch.int32, device="cuda")
                    self.h.sparse_decode(layer, self.caches[layer], self.pools[layer][2], q, k, v, self.pos, o, self.num,
                                         gate=gate, write_back=False, selected=sel)
                    done(o, sel)
                elif kind == "d":
                    self.h.decode(layer, self.caches[layer], q, k, v, self.pos, o, gate=gate, write_back=False)
                    done(o)
                else:
                    out = torch.zeros(4, 500, 8, 256, device="cuda")
                    self.h.prefill(2, cache, *self.prompt[:3], self.counts, self.zero, out, gate=self.prompt[3])
                    done(out)
                    self.h.decode(2, cache, q, k, v, self.pos, o, gate=gate)
                    done(o)
        outs.append(state)
        return outs


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_calls_behind_one_another(dattn):
    m = Mixed(dattn, 71)
    want = m.calls(True)
    assert m.h.get_error() == dattn.OK and all(torch.isfinite(x.float()).all() for x in want)
    for _ in range(5):
        same(m.calls(False), want)
    assert m.h.get_error() == dattn.OK


def test_two_handles_on_two_streams(dattn):
    ms = [Mixed(dattn, 72), Mixed(dattn, 73)]
    want = [m.calls(True) for m in ms]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for m, s in zip(ms, streams):
            with torch.cuda.stream(s):
                got.append(m.calls(False))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        same(x, want[i % 2])
    for m, s in zip(ms, streams):
        assert m.h.get_error(s) == dattn.OK


def test_captured_and_replayed(dattn):
    m = Mixed(dattn, 74)
    want = m.calls(True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            got = m.calls(False)
        for _ in range(3):
            graph.replay()
            stream.synchronize()
            same(got, want)
    assert m.h.get_error(stream) == dattn.OK
