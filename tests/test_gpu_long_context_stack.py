"""A small stack as a model would run it: a layer that attends over selected
pages and a layer with a recurrent state, prompts in one call each, then decode
steps - the first ones eager, the rest replayed from one graph on a side stream.

Every step is compared with 64 bits: the page summaries with the means of the
stored keys (half a bf16 step, and P fp32 roundings of the mean absolute key),
the selection page for page with the scores of the summaries as stored, the
attention over the selected pages' stored entries within the decode tolerance,
the state layer with the recurrence (per element: the prompt form's
2^-16 + (D + 128) 2^-23 of the sum of the contributions' sizes, and 2^-23 more a step).
"""
import pytest
import torch

from gpu_util import assert_close
from test_gpu_linear import Ref, close, decays
from test_gpu_sparse import rotate

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


class Stack:
    def __init__(self, dattn, seed, Hq, Hkv, D, P, count, steps, num, fp8):
        self.d, self.Hq, self.Hkv, self.D, self.P, self.count, self.num = dattn, Hq, Hkv, D, P, count, num
        self.g = torch.Generator().manual_seed(seed)
        self.first, self.last, self.r, self.theta = 1, 2, D // 4, 1e4
        self.ks, self.vs = (0.75, 1.25) if fp8 else (1.0, 1.0)
        B = self.B = len(count)
        kind = F8 if fp8 else torch.bfloat16
        width = max(-(-(n + steps) // P) for n in count)
        pages = B * width + 1
        self.table = torch.randperm(pages, generator=self.g)[:B * width].view(B, width).int()
        self.k = torch.full((pages, Hkv, P, D), float("nan")).to(kind).cuda()
        self.v = self.k.clone()
        self.summary = torch.full((pages, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.state = torch.randn(B + 1, Hkv, D, D, generator=self.g)
        self.rows = torch.arange(B, 0, -1, dtype=torch.int32)  # (row 0 belongs to none)
        self.ref = Ref(self.state, decays(Hkv))
        self.sd = self.state.cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.td, self.rd, self.len, self.pos = self.table.cuda(), self.rows.cuda(), i32([0] * B), i32([0] * B)
        paged = {"kind": dattn.CACHE_PAGED, "page_size": P, "rotary_dim": self.r, "rope_theta": self.theta}
        if fp8:
            paged.update(kv_format=dattn.KV_E4M3, k_scale=self.ks, v_scale=self.vs)
        self.h = dattn.Handle(Hq, Hkv, D, [paged, {"kind": dattn.CACHE_STATE, "log_decay": decays(Hkv)}], B,
                              max_context=width * P, max_selected_pages=num)
        self.paged = dattn.paged_cache(self.k, self.v, self.td, self.len)
        self.st = dattn.state_cache(self.sd, self.rd)
        self.eps = 2.0 ** -16 + (D + 128) * 2.0 ** -23
        self.steps = 0

    def inputs(self, *lead):
        rn = lambda *s: torch.randn(*s, generator=self.g).to(torch.bfloat16)  # noqa: E731
        return [rn(*lead, self.Hq, self.D), rn(*lead, self.Hkv, self.D), rn(*lead, self.Hkv, self.D), rn(*lead, self.Hq)]

    def prompt(self):
        T = max(self.count)
        x, y = self.inputs(self.B, T), self.inputs(self.B, T)
        for b, n in enumerate(self.count):
            for t in x + y:
                t[b, n:] = float("nan")
        n = torch.tensor(self.count, dtype=torch.int32).cuda()
        zero = torch.zeros_like(n)
        xd, yd = [t.cuda() for t in x], [t.cuda() for t in y]
        out = torch.full((self.B, T, self.Hq, self.D), 7.0, device="cuda")
        self.h.append_kv(0, self.paged, xd[1], xd[2], zero, n, start_pos=zero)
        self.len.copy_(n)
        self.pos.copy_(n)
        self.h.summarize(0, self.paged, self.summary, zero, n, T)
        self.h.prefill(1, self.st, *yd[:3], n, zero, out, gate=yd[3])
        assert self.h.get_error() == self.d.OK
        out = out.cpu()
        for b, n in enumerate(self.count):
            for t in range(n):
                want, size = self.ref.step(int(self.rows[b]), y[0][b, t], y[1][b, t], y[2][b, t], y[3][b, t])
                close(out[b, t], want, size, self.eps, f"prompt row {b} token {t}")
            assert (out[b, n:] == 7.0).all()

    def buffers(self):
        B, Hq, D = self.B, self.Hq, self.D
        self.x, self.y = [t.cuda() for t in self.inputs(B)], [t.cuda() for t in self.inputs(B)]
        self.o0, self.o1 = torch.empty(B, Hq, D, device="cuda"), torch.empty(B, Hq, D, device="cuda")
        self.sel = torch.empty(B, self.Hkv, self.num, dtype=torch.int32, device="cuda")
        self.one = torch.ones(B, dtype=torch.int32, device="cuda")

    def step(self):
        """One token through both layers; the metadata moves on in the stream."""
        x, y = self.x, self.y
        self.h.sparse_decode(0, self.paged, self.summary, *x[:3], self.pos, self.o0, self.num, keep_first=self.first,
                             keep_last=self.last, gate=x[3], selected=self.sel)
        self.h.decode(1, self.st, *y[:3], self.pos, self.o1, gate=y[3])
        self.h.summarize(0, self.paged, self.summary, self.len, self.one, 1)
        self.len += 1
        self.pos += 1

    def check(self, k, v, summary, lens):
        """The step just run against the pools and summaries as they were before it."""
        P, G, D = self.P, self.Hq // self.Hkv, self.D
        x, y = [t.cpu() for t in self.x], [t.cpu() for t in self.y]
        sel = self.sel.cpu()
        want = torch.empty(self.B, self.Hq, D, dtype=torch.float64)
        k1, v1, s1 = (t.cpu().double() for t in (self.k, self.v, self.summary))
        for b, n in enumerate(lens):
            pages = -(-n // P)
            for h in range(self.Hkv):
                q = rotate(x[0][b, h * G:(h + 1) * G].double(), n, self.r, self.theta)
                pick = list(range(pages))
                if pages > self.num:
                    s = (q[None] * summary[self.table[b, :pages].long(), h][:, None]).sum(-1).amax(1)
                    sure = [p for p in pick if p < self.first or p >= pages - self.last]
                    rest = sorted((p for p in pick if p not in sure), key=lambda p: (-float(s[p]), p))
                    pick = sorted(sure + rest[:self.num - len(sure)])
                assert sel[b, h].tolist() == pick + [-1] * (self.num - len(pick)), (b, h)
                # the new entry as the step stored it
                row, slot = int(self.table[b, n // P]), n % P
                kk = [k[int(self.table[b, p]), h, :min(P, n - p * P)] for p in pick] + [k1[row, h, slot][None]]
                vv = [v[int(self.table[b, p]), h, :min(P, n - p * P)] for p in pick] + [v1[row, h, slot][None]]
                a = torch.softmax(q @ (torch.cat(kk) * self.ks).T / D ** 0.5, -1) @ (torch.cat(vv) * self.vs)
                want[b, h * G:(h + 1) * G] = a / (1 + torch.exp(-x[3][b, h * G:(h + 1) * G].double()))[:, None]
                if slot == P - 1:  # the step completed the page
                    key = k1[row, h] * self.ks
                    mean = key.mean(0)
                    bound = 2.0 ** -8 * mean.abs() + (P + 1) * 2.0 ** -24 * key.abs().mean(0) + 2.0 ** -130
                    assert ((s1[row, h] - mean).abs() <= bound).all(), (b, h)
        assert_close(self.o0.cpu().numpy(), want.numpy())
        o1 = self.o1.cpu()
        for b in range(self.B):
            w, size = self.ref.step(int(self.rows[b]), y[0][b], y[1][b], y[2][b], y[3][b])
            close(o1[b], w, size, self.eps + self.steps * 2.0 ** -23, f"state layer, step {self.steps} row {b}")
        self.steps += 1

    def before(self):
        return [t.cpu().double() for t in (self.k, self.v, self.summary)], self.len.tolist()

    def refresh(self):
        for old, new in zip(self.x + self.y, self.inputs(self.B) + self.inputs(self.B)):
            old.copy_(new)


@pytest.mark.parametrize("Hq,Hkv,D,P,fp8", [(8, 2, 256, 8, False), (16, 8, 128, 16, False), (6, 2, 128, 5, True)])
def test_prompts_then_steps(dattn, Hq, Hkv, D, P, fp8):
    steps = 14
    s = Stack(dattn, Hq + D + P, Hq, Hkv, D, P, [20 * P + 5, 3, 9 * P - 1, 0], steps, 6, fp8)
    s.prompt()
    s.buffers()
    for _ in range(2):
        was, lens = s.before()
        s.step()
        assert s.h.get_error() == dattn.OK
        s.check(*was, lens)
        s.refresh()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            s.step()
        for _ in range(steps - 2):
            was, lens = s.before()
            graph.replay()
            stream.synchronize()
            s.check(*was, lens)
            s.refresh()
    assert s.h.get_error(stream) == dattn.OK
    # the row of no stream, and the states of the others
    state = s.sd.cpu()
    assert torch.equal(state[0], s.state[0])
    close(state, s.ref.s, s.ref.a, s.eps + steps * 2.0 ** -23, "states")
