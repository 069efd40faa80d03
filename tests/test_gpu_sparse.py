"""Decode over selected pages and the page summaries it scores, on the GPU.

The selection is compared page for page with the selection of the scores in
64 bits (ties to the lower page); the outputs with attention in 64 bits over
the selected tokens, within the decode tolerance; every page that is not
selected holds NaN, so that a read of one shows. Summaries: the fp32 sum of P
keys and a bf16 rounding, so within half a bf16 step (2^-8) of the exact mean
plus P fp32 roundings of the mean absolute key.
"""
import numpy as np
import pytest
import torch

import synth
from gpu_util import assert_close, dev, host_u16

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def rotate(x, pos, r, theta):
    """x [..., D] float64, the first r dims turned at pos, in 64 bits."""
    half = r // 2
    if not half:
        return x.clone()
    a = pos * theta ** (-torch.arange(half, dtype=torch.float64) * 2 / r)
    c, s = a.cos(), a.sin()
    y = x.clone()
    y[..., :half] = x[..., :half] * c - x[..., half:r] * s
    y[..., half:r] = x[..., half:r] * c + x[..., :half] * s
    return y


def norm(x, w, eps):
    if w is None:
        return x
    return (w.double() * x.double() / (x.double().pow(2).mean(-1, keepdim=True) + eps).sqrt()).to(torch.bfloat16)


class Case:
    """A paged cache with exact bf16 (or E4M3) values on the host."""

    def __init__(self, seed, Hq, Hkv, D, P, lens, fp8=False, r=64, theta=5e6, gate=True, qk_norm=False, q_mul=1.0,
                 spread=0.5):
        g = self.g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.P, self.lens, self.fp8, self.r, self.theta = Hq, Hkv, D, P, lens, fp8, r, theta
        B = len(lens)
        rn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
        need = [n // P + 1 for n in lens]
        total = sum(need) + 2
        perm = torch.randperm(total, generator=g)
        self.width = max(need)
        self.table = torch.full((B, self.width), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m].int()
            at += m
        k = torch.randn(total, Hkv, P, D, generator=g) + spread * torch.randn(total, Hkv, 1, D, generator=g)
        v = torch.randn(total, Hkv, P, D, generator=g)
        self.kind = F8 if fp8 else torch.bfloat16
        self.k, self.v = k.to(self.kind), v.to(self.kind)
        self.ks, self.vs = (0.625, 1.5) if fp8 else (1.0, 1.0)
        self.q, self.k_new, self.v_new = (rn(B, Hq, D).float() * q_mul).to(torch.bfloat16), rn(B, Hkv, D), rn(B, Hkv, D)
        self.gate = rn(B, Hq) if gate else None
        self.pos = torch.tensor(lens, dtype=torch.int32)
        self.wq = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if qk_norm else None
        self.wk = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if qk_norm else None
        self.eps = 1e-6
        self.summary = (self.k.float().mean(2) * self.ks).to(torch.bfloat16)

    def layer(self, dattn):
        L = {"kind": dattn.CACHE_PAGED, "page_size": self.P, "rotary_dim": self.r, "rope_theta": self.theta}
        if self.fp8:
            L.update(kv_format=dattn.KV_E4M3, k_scale=self.ks, v_scale=self.vs)
        if self.wq is not None:
            L.update(q_norm=self.wq, k_norm=self.wk, norm_eps=self.eps)
        return L

    def rotated(self, b, h):
        G = self.Hq // self.Hkv
        return rotate(norm(self.q[b, h * G:(h + 1) * G], self.wq, self.eps).double(), int(self.pos[b]), self.r, self.theta)

    def selection(self, num, first, last):
        B = len(self.lens)
        out = torch.full((B, self.Hkv, num), -1, dtype=torch.int32)
        for b, n in enumerate(self.lens):
            m = -(-n // self.P)
            for h in range(self.Hkv):
                pick = list(range(m))
                if m > num:
                    rows = self.table[b, :m].long()
                    prod = self.rotated(b, h)[None] * self.summary[rows, h].double()[:, None]
                    s = prod.sum(-1)
                    s = torch.where(s != s, torch.inf, s).amax(1).tolist()
                    sure = [p for p in range(m) if p < first or p >= m - last]
                    rest = sorted((p for p in range(m) if first <= p < m - last), key=lambda p: (-s[p], p))
                    pick = sorted(sure + rest[:num - len(sure)])
                out[b, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
        return out

    def entries(self, b, h):
        """The new K and V entries as they are stored."""
        k = rotate(norm(self.k_new[b, h], self.wk, self.eps).double(), int(self.pos[b]), self.r, self.theta)
        k, v = k.to(torch.bfloat16), self.v_new[b, h]
        if self.fp8:
            k = (k.double() / self.ks).clamp(-448, 448).float().to(F8)
            v = (v.double() / self.vs).clamp(-448, 448).float().to(F8)
        return k, v

    def attention(self, selected):
        B, G = len(self.lens), self.Hq // self.Hkv
        out = torch.empty(B, self.Hq, self.D, dtype=torch.float64)
        for b, n in enumerate(self.lens):
            for h in range(self.Hkv):
                pages = [int(p) for p in selected[b, h] if p >= 0]
                kk = [self.k[int(self.table[b, p]), h, :min(self.P, n - p * self.P)].double() * self.ks for p in pages]
                vv = [self.v[int(self.table[b, p]), h, :min(self.P, n - p * self.P)].double() * self.vs for p in pages]
                k1, v1 = self.entries(b, h)
                kk, vv = torch.cat(kk + [k1.double()[None] * self.ks]), torch.cat(vv + [v1.double()[None] * self.vs])
                a = torch.softmax(self.rotated(b, h) @ kk.T / self.D ** 0.5, -1) @ vv
                out[b, h * G:(h + 1) * G] = a
        if self.gate is not None:
            out /= 1 + torch.exp(-self.gate.double())[..., None]
        return out

    def poison(self, selected):
        """The pools with NaN in every (page, head) that is not selected and in every slot past a length."""
        k, v = self.k.float(), self.v.float()
        keep = torch.zeros(k.shape[:3], dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for h in range(self.Hkv):
                for p in selected[b, h]:
                    if p >= 0:
                        keep[int(self.table[b, p]), h, :max(0, min(self.P, n - int(p) * self.P))] = True
        k[~keep] = float("nan")
        v[~keep] = float("nan")
        return k.to(self.kind), v.to(self.kind)

    def handle(self, dattn, num, max_context=None):
        return dattn.Handle(self.Hq, self.Hkv, self.D, [self.layer(dattn)], len(self.lens),
                            max_context=max_context or max(max(self.lens), 1), max_selected_pages=num)

    def run(self, dattn, num, first, last, write=False, k=None, v=None, handle=None, expect=None):
        h = handle or self.handle(dattn, num)
        self.kd, self.vd = (self.k if k is None else k).cuda(), (self.v if v is None else v).cuda()
        d = lambda x: None if x is None else x.cuda()  # noqa: E731
        self.td, self.nd = self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        cache = dattn.paged_cache(self.kd, self.vd, self.td, self.nd)
        out = torch.full((len(self.lens), self.Hq, self.D), float("nan"), device="cuda")
        sel = torch.full((len(self.lens), self.Hkv, num), -7, dtype=torch.int32, device="cuda")
        h.sparse_decode(0, cache, self.summary.cuda(), d(self.q), d(self.k_new), d(self.v_new), d(self.pos), out, num,
                        keep_first=first, keep_last=last, gate=d(self.gate), write_back=write, selected=sel)
        status = h.get_error()
        assert status == (dattn.OK if expect is None else expect)
        return out.cpu(), sel.cpu()


LAYOUTS = [(8, 2, 256, 16), (16, 8, 128, 16), (24, 4, 256, 16), (4, 4, 128, 24), (5, 1, 128, 40), (3, 1, 256, 7),
           (16, 2, 128, 64), (6, 2, 128, 1)]


@pytest.mark.parametrize("Hq,Hkv,D,P", LAYOUTS)
@pytest.mark.parametrize("fp8", [False, True])
def test_selection_and_output(dattn, Hq, Hkv, D, P, fp8):
    num, first, last = 9, 1, 2
    lens = [0, 1, P, max(1, P - 1), P + 1, num * P, num * P + 1, 40 * P, 57 * P + 3 % P, 33 * P - 1]
    c = Case(Hq * D + P, Hq, Hkv, D, P, lens, fp8=fp8, r=D // 4 if P != 24 else D)
    want = c.selection(num, first, last)
    out, sel = c.run(dattn, num, first, last, k=c.poison(want)[0], v=c.poison(want)[1])
    assert torch.equal(sel, want)
    assert_close(out.numpy(), c.attention(want).numpy())


@pytest.mark.parametrize("num,first,last", [(1, 0, 1), (3, 1, 2), (3, 0, 1), (64, 4, 8), (200, 0, 1), (40, 39, 1)])
def test_budgets(dattn, num, first, last):
    """From the newest page alone to more pages than any stream has; nothing left to choose where the kept pages
    fill the budget."""
    c = Case(5, 8, 2, 128, 16, [16 * 150 + 5, 16 * 64, 700, 15], r=128, theta=1e6, gate=False)
    want = c.selection(num, first, last)
    out, sel = c.run(dattn, num, first, last, k=c.poison(want)[0], v=c.poison(want)[1])
    assert torch.equal(sel, want)
    assert_close(out.numpy(), c.attention(want).numpy())


def test_long_streams(dattn):
    """Thousands of pages, several score CTAs a unit, and the threshold search over all of them."""
    c = Case(11, 8, 1, 128, 16, [16 * 9000 + 1, 16 * 130, 16 * 2049], r=32, gate=False)
    want = c.selection(48, 1, 2)
    out, sel = c.run(dattn, 48, 1, 2)
    assert torch.equal(sel, want)
    assert_close(out.numpy(), c.attention(want).numpy())


def test_qk_norm(dattn):
    c = Case(12, 8, 2, 256, 16, [900, 2000], qk_norm=True)
    want = c.selection(12, 1, 1)
    out, sel = c.run(dattn, 12, 1, 1)
    assert torch.equal(sel, want)
    assert_close(out.numpy(), c.attention(want).numpy())


@pytest.mark.parametrize("pages", [60, 1500])
def test_equal_scores_take_the_lower_page(dattn, pages):
    """Every summary alike, then two alternating ones: few and very many pages at the border."""
    c = Case(13, 8, 2, 128, 16, [16 * pages])
    c.summary[:] = c.summary[:1]
    want = c.selection(20, 1, 1)
    assert want[0, 0, :19].tolist() == list(range(19))
    assert torch.equal(c.run(dattn, 20, 1, 1)[1], want)
    c.summary[c.table[0, 1::2].long()] = c.summary[c.table[0, 0].long()] * 2
    assert torch.equal(c.run(dattn, 20, 1, 1)[1], c.selection(20, 1, 1))


def test_scores_that_32_bits_cannot_tell_apart(dattn):
    """Summaries whose large terms cancel: the pages differ by less than an fp32 sum keeps."""
    c = Case(14, 4, 2, 128, 16, [16 * 200], r=0)
    c.q[:] = 1.0
    c.q[..., 0] = 2.0
    s = torch.zeros_like(c.summary)
    s[..., 0], s[..., 1] = 2.0 ** 20, -(2.0 ** 21)
    order = torch.randperm(s.shape[0], generator=c.g)
    s[..., 2] = (order[:, None] - s.shape[0] // 2).float().to(torch.bfloat16) * 2.0 ** -12
    c.summary = s
    want = c.selection(16, 1, 1)
    assert torch.equal(c.run(dattn, 16, 1, 1)[1], want)


@pytest.mark.parametrize("what", ["nan", "inf", "-inf", "large", "small", "nan query", "zero"])
def test_values_beyond_the_screen(dattn, what):
    """No numbers, infinities, sums beyond the fp32 range and below it, in summaries that compete. The keys themselves
    stay finite, so the output does."""
    c = Case(15, 8, 2, 128, 16, [16 * 90, 16 * 1300], r=64)
    rows = c.table[:, 3:40:5].reshape(-1).long()
    if what in ("nan", "inf", "-inf"):
        c.summary[rows, :, 5] = float(what)
    elif what == "large":
        c.summary = (c.summary.float() * 2.0 ** 125).to(torch.bfloat16)
        c.q = (c.q.float() * 2.0 ** 60).to(torch.bfloat16)
    elif what == "small":
        c.summary = (c.summary.float() * 2.0 ** -70).to(torch.bfloat16)
        c.q = (c.q.float() * 2.0 ** -70).to(torch.bfloat16)
    elif what == "zero":
        c.summary[:] = 0
    else:
        c.q[0, 1, 3] = float("nan")
    want = c.selection(12, 1, 2)
    out, sel = c.run(dattn, 12, 1, 2)
    assert torch.equal(sel, want)
    if what in ("nan", "inf", "-inf", "zero"):
        assert_close(out.numpy(), c.attention(want).numpy())


@pytest.mark.parametrize("fp8", [False, True])
def test_write_back(dattn, fp8):
    """The new entries land in their slots - a page's middle, its last slot, a page of its own - and nothing else
    changes; without write-back nothing does."""
    c = Case(16, 8, 2, 128, 16, [16 * 30 + 7, 16 * 30 + 15, 16 * 30, 5, 0, 16], fp8=fp8)
    bits = lambda t: t.cpu().view(torch.uint8 if fp8 else torch.int16)  # noqa: E731
    k, v = bits(c.k).clone(), bits(c.v).clone()
    c.run(dattn, 8, 1, 2, write=False)
    assert torch.equal(bits(c.kd), k) and torch.equal(bits(c.vd), v)
    c.run(dattn, 8, 1, 2, write=True)
    for b, n in enumerate(c.lens):
        pg = int(c.table[b, n // 16])
        for h in range(2):
            k1, v1 = c.entries(b, h)
            k[pg, h, n % 16], v[pg, h, n % 16] = bits(k1), bits(v1)
    assert torch.equal(bits(c.kd), k) and torch.equal(bits(c.vd), v)


def test_selection_matches_decode_when_every_page_fits(dattn):
    """With no fewer pages than a stream has, the outputs are those of dattn_decode."""
    c = Case(17, 16, 8, 128, 16, [300, 77, 1, 0])
    out, sel = c.run(dattn, 32, 1, 1)
    h = c.handle(dattn, 32)
    ref = torch.empty_like(out, device="cuda")
    h.decode(0, dattn.paged_cache(c.kd, c.vd, c.td, c.nd), c.q.cuda(), c.k_new.cuda(), c.v_new.cuda(), c.pos.cuda(),
             ref, gate=c.gate.cuda(), write_back=False)
    assert h.get_error() == dattn.OK
    assert_close(out.numpy(), ref.cpu().numpy())


def test_bad_metadata_is_reported(dattn):
    c = Case(18, 8, 2, 128, 16, [16 * 40, 16 * 50])
    c.table[0, 7] = 10 ** 6
    c.run(dattn, 8, 1, 1, expect=dattn.EINDEX)
    c.table[0, 7] = -1
    c.run(dattn, 8, 1, 1, expect=dattn.EINDEX)
    c = Case(18, 8, 2, 128, 16, [16 * 40, 16 * 50])
    h = c.handle(dattn, 8, max_context=16 * 45)
    c.run(dattn, 8, 1, 1, handle=h, expect=dattn.ELENGTH)
    c.lens[1] = -3
    c.run(dattn, 8, 1, 1, handle=h, expect=dattn.ELENGTH)
    c.lens[1] = 16 * 44
    assert torch.equal(c.run(dattn, 8, 1, 1, handle=h)[1], c.selection(8, 1, 1))


def test_refusals(dattn):
    c = Case(19, 8, 2, 128, 16, [100])
    h = dattn.Handle(8, 2, 128, [c.layer(dattn), {"kind": dattn.CACHE_RING, "ring_slots": 33}], 1, max_context=128,
                     max_selected_pages=8)
    kd, td, nd = c.k.cuda(), c.table.cuda(), torch.tensor([100], dtype=torch.int32).cuda()
    cache = dattn.paged_cache(kd, kd, td, nd)
    x = [c.q.cuda(), c.k_new.cuda(), c.v_new.cuda(), c.pos.cuda(), torch.empty(1, 8, 128, device="cuda")]
    s = c.summary.cuda()

    def refused(code, num, first, last, layer=0, cache=cache, summary=s, handle=h, **kw):
        with pytest.raises(dattn.DattnError) as e:
            handle.sparse_decode(layer, cache, summary, *x, num, keep_first=first, keep_last=last, **kw)
        assert e.value.code == code

    refused(dattn.EXCEEDS, 9, 1, 1)
    refused(dattn.EINVAL, 0, 0, 1)
    refused(dattn.EINVAL, 4, 0, 0)
    refused(dattn.EINVAL, 4, -1, 1)
    refused(dattn.EINVAL, 4, 3, 2)
    refused(dattn.EINVAL, 4, 2 ** 31 - 1, 1)
    refused(dattn.EXCEEDS, 4, 1, 1, max_seq_len=129)
    refused(dattn.EINVAL, 4, 1, 1, summary=None)
    ring = dattn.ring_cache(kd, kd, nd, nd)
    refused(dattn.EUNSUPPORTED, 4, 1, 1, layer=1, cache=ring)
    refused(dattn.EXCEEDS, 1, 0, 1, handle=dattn.Handle(8, 2, 128, [c.layer(dattn)], 1, max_context=128))
    with pytest.raises(dattn.DattnError) as e:
        h.summarize(1, ring, s, nd, nd, max_tokens=4)
    assert e.value.code == dattn.EUNSUPPORTED
    with pytest.raises(dattn.DattnError) as e:
        h.summarize(0, cache, s, nd, nd, max_tokens=-1)
    assert e.value.code == dattn.EINVAL
    h.summarize(0, cache, s, nd, nd, max_tokens=0)
    assert h.get_error() == dattn.OK


# ---------------------------------------------------------------- summaries

@pytest.mark.parametrize("Hkv,D,P", [(2, 256, 16), (8, 128, 16), (1, 128, 24), (4, 256, 64), (1, 256, 7), (3, 128, 1),
                                     (2, 128, 130)])
@pytest.mark.parametrize("fp8", [False, True])
def test_summaries(dattn, Hkv, D, P, fp8):
    """Only the pages that the new tokens complete are written, from their keys alone."""
    lens = [0, 1, P, 5 * P, 5 * P + P // 2, 9 * P - 1, 12 * P]
    start = [0, 0, 0, 2 * P, 3 * P - 1, 4 * P, 12 * P]
    count = [0, 1, P, 3 * P, 2 * P + 1 + P // 2, 5 * P - 1, 0]
    c = Case(D + P, Hkv, Hkv, D, P, lens, fp8=fp8)
    h = c.handle(dattn, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    # tokens that are not written yet are NaN: a summary reads full pages only
    k = c.k.float()
    for b, n in enumerate(lens):
        if n % P:
            k[int(c.table[b, n // P]), :, n % P:] = float("nan")
    kd = k.to(c.kind).cuda()
    s = torch.full((kd.shape[0], Hkv, D), -5.0, dtype=torch.bfloat16, device="cuda")
    cache = dattn.paged_cache(kd, kd, c.table.cuda(), i32(lens))
    h.summarize(0, cache, s, i32(start), i32(count), max_tokens=max(count))
    assert h.get_error() == dattn.OK
    got = s.cpu().double()
    done = set()
    for b in range(len(lens)):
        for p in range(start[b] // P, (start[b] + count[b]) // P):
            done.add(int(c.table[b, p]))
    for pg in range(kd.shape[0]):
        if pg not in done:
            assert (got[pg] == -5.0).all()
            continue
        keys = c.k[pg].double() * c.ks
        mean, size = keys.mean(1), keys.abs().mean(1)
        assert ((got[pg] - mean).abs() <= mean.abs() * 2.0 ** -8 + size * (P + 2) * 2.0 ** -24).all()


def test_summaries_report_bad_metadata(dattn):
    c = Case(20, 8, 2, 128, 16, [16 * 10])
    h = c.handle(dattn, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    kd = c.k.cuda()
    s = torch.full((kd.shape[0], 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    cache = dattn.paged_cache(kd, kd, c.table.cuda(), i32([160]))
    for start, count, most in (([0], [-1], 8), ([0], [33], 32), ([-1], [16], 32), ([2 ** 31 - 8], [16], 32), ([160], [32], 32)):
        h.summarize(0, cache, s, i32(start), i32(count), max_tokens=most)
        assert h.get_error() == dattn.EINDEX
    assert (s[c.table[0, :10].long().cuda()] == 3.0).all()


# ---------------------------------------------------------------- use

def test_other_stream_and_graph_replay(dattn):
    """Captured on a side stream and replayed with new queries; another handle's calls between."""
    c = Case(21, 8, 2, 256, 16, [16 * 70 + 3, 16 * 33])
    num = 12
    h, other = c.handle(dattn, num), c.handle(dattn, num)
    kd, vd, sd, td = c.k.cuda(), c.v.cuda(), c.summary.cuda(), c.table.cuda()
    nd, pd = torch.tensor(c.lens, dtype=torch.int32).cuda(), c.pos.cuda()
    cache = dattn.paged_cache(kd, vd, td, nd)
    q, kn, vn, g = c.q.cuda(), c.k_new.cuda(), c.v_new.cuda(), c.gate.cuda()
    out = torch.empty(2, 8, 256, device="cuda")
    sel = torch.empty(2, 2, num, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    args = (0, cache, sd, q, kn, vn, pd, out, num)
    with torch.cuda.stream(stream):
        h.sparse_decode(*args, gate=g, write_back=False, selected=sel)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            h.sparse_decode(*args, gate=g, write_back=False, selected=sel)
            h.sparse_decode(*args, gate=g, write_back=False, selected=sel)
        for i in range(3):
            c.q = torch.randn(2, 8, 256, generator=c.g).to(torch.bfloat16)
            q.copy_(c.q)
            out.fill_(float("nan"))
            graph.replay()
            other_out = torch.empty_like(out)
            other.sparse_decode(0, cache, sd, q, kn, vn, pd, other_out, num, gate=g, write_back=False)
            stream.synchronize()
            want = c.selection(num, 1, 1)
            assert torch.equal(sel.cpu(), want)
            assert_close(out.cpu().numpy(), c.attention(want).numpy())
            assert torch.equal(other_out, out)
    assert h.get_error() == dattn.OK and other.get_error() == dattn.OK


def test_same_inputs_give_the_same_bits(dattn):
    c = Case(22, 16, 8, 128, 16, [16 * 100 + 9] * 4)
    first = c.run(dattn, 24, 1, 2)
    for _ in range(3):
        again = c.run(dattn, 24, 1, 2)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
