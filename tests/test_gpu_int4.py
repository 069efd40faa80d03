"""The 4-bit cache on the GPU against 64-bit arithmetic (int4_ref.py; QK-norms from the
oracle): append, read back, decode, and runs of them together.

Written bytes are compared bit for bit, and so is everything beside them. Decode
outputs: with the cache's values given, what differs from 64 bits is q (two fp16 terms:
2^-22 of each dim's product), fp32 sums of D products (taken as a walk of D roundings of
2^-24, four times its expected size) and the weights; a score that is off by e moves an
output by at most 2 e of the largest value, and the outputs' own sums add 2^-20 of it.
"""
import numpy as np
import pytest
import torch

import int4_ref as ref
import synth
from gpu_util import dev, host_u16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def tables(rng, lens, P, room=1, spare=3):
    """Page table of streams with room for their lengths and `room` more tokens, and the pool's size."""
    pages = [(max(n, 0) + room + P - 1) // P for n in lens]
    total = sum(pages) + spare
    perm, nxt = rng.permutation(total).astype(np.int32), 0
    bt = np.full((len(lens), max(pages)), -1, np.int32)
    for b, n in enumerate(pages):
        bt[b, :n] = perm[nxt:nxt + n]
        nxt += n
    return bt, total


def entries(rng, *shape):
    """bf16 bits: dims of unlike spread, some off zero."""
    x = rng.standard_normal(shape) * (0.5 + np.arange(shape[-1]) % 5 / 2) + (np.arange(shape[-1]) % 13 == 0) * 3
    return ref.bf16_bits(x)


class Case:
    def __init__(self, seed, Hq, Hkv, D, P, lens, rope=(0, 0.0), gate=False, norm=False, q_mul=1.0, make=entries, room=1):
        self.rng = rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D, self.P, self.lens, self.rope = Hq, Hkv, D, P, list(lens), rope
        B = len(lens)
        self.bt, self.pages = tables(rng, lens, P, room)
        self.pool = {s: ref.random_pool(rng, self.pages, Hkv, P, D) for s in "kv"}
        self.values = {s: [] for s in "kv"}
        for b, n in enumerate(lens):
            for s in "kv":
                x = ref.f64(make(rng, max(n, 0), Hkv, D))
                code, lo, st = ref.quantise(x)
                for t in range(n):
                    ref.store(self.pool[s], s, self.bt[b, t // P], t % P, code[t], lo[t], st[t])
                self.values[s].append(ref.value(code, lo, st))  # [n, H, D]
        self.q = ref.bf16_bits(rng.standard_normal((B, Hq, D)) * q_mul)
        self.k_new, self.v_new = entries(rng, B, Hkv, D), entries(rng, B, Hkv, D)
        self.gate = ref.bf16_bits(rng.standard_normal((B, Hq))) if gate else None
        self.pos = np.array([max(n, 0) for n in lens], np.int32)
        self.norm = (ref.bf16_bits(1 + 0.25 * rng.standard_normal(D)), ref.bf16_bits(1 + 0.25 * rng.standard_normal(D)),
                     1e-6) if norm else None

    def layer(self, dattn):
        l = {"kind": dattn.CACHE_PAGED, "page_size": self.P, "rotary_dim": self.rope[0], "rope_theta": self.rope[1],
             "kv_format": dattn.KV_INT4}
        if self.norm:
            l.update(q_norm=self.norm[0], k_norm=self.norm[1], norm_eps=self.norm[2])
        return l

    def handle(self, dattn, max_context=None, **kw):
        return dattn.Handle(self.Hq, self.Hkv, self.D, [self.layer(dattn)], len(self.lens),
                            max_context=max_context or max(max(self.lens), 1), **kw)

    def upload(self, dattn):
        self.dev = {s: dev(self.pool[s]) for s in "kv"}
        self.keep = (dev(self.bt), dev(np.array(self.lens, np.int32)))
        return dattn.paged_cache(self.dev["k"], self.dev["v"], *self.keep)

    def entry(self, oracle, x, pos, rotate=True):
        """A key head's entry: normalised, and turned in 64 bits, rounded to bf16 by way of fp32."""
        if rotate and self.norm:
            x = oracle.qk_norm(x, self.norm[1], self.norm[2])
        if rotate and self.rope[0]:
            x = ref.bf16_bits(ref.rotate(ref.f64(x), self.rope[0], self.rope[1], int(pos)))
        return x

    def new(self, oracle, b):
        """Stream b's new token as it is stored: (code, least, step) of K and V."""
        k = np.stack([self.entry(oracle, self.k_new[b, j], self.pos[b]) for j in range(self.Hkv)])
        return ref.quantise(ref.f64(k)), ref.quantise(ref.f64(self.v_new[b]))

    def query(self, oracle, b, h):
        x = oracle.qk_norm(self.q[b, h], self.norm[0], self.norm[2]) if self.norm else self.q[b, h]
        return ref.rotate(ref.f64(x), *self.rope, int(self.pos[b])) if self.rope[0] else ref.f64(x)

    def expect(self, oracle, write, bound=None):
        """Outputs, tolerance of each stream, pools afterwards."""
        B, G, D = len(self.lens), self.Hq // self.Hkv, self.D
        out, tol = np.empty((B, self.Hq, D)), np.empty((B, self.Hq, 1))
        pool = {s: self.pool[s].copy() for s in "kv"}
        for b in range(B):
            nk, nv = self.new(oracle, b)
            n = self.lens[b] if bound is None else min(self.lens[b], bound)
            for j in range(self.Hkv):
                k = np.concatenate([self.values["k"][b][:n, j], ref.value(*nk)[j:j + 1]])
                v = np.concatenate([self.values["v"][b][:n, j], ref.value(*nv)[j:j + 1]])
                q = np.stack([self.query(oracle, b, j * G + i) for i in range(G)])
                gate = None if self.gate is None else ref.f64(self.gate[b, j * G:(j + 1) * G])
                out[b, j * G:(j + 1) * G] = ref.attend(q, k, v, D ** -0.5, gate)
                e = (2.0 ** -22 + 4 * D ** 0.5 * 2.0 ** -24) * (np.abs(q) @ np.abs(k).T).max(-1) / D ** 0.5
                tol[b, j * G:(j + 1) * G, 0] = (2 * e + 2.0 ** -20) * np.abs(v).max()
            if write and n == self.lens[b]:
                at = self.bt[b, n // self.P], n % self.P
                ref.store(pool["k"], "k", *at, *nk)
                ref.store(pool["v"], "v", *at, *nv)
        return out, tol, pool

    def check(self, dattn, oracle, write=True, max_context=None, **kw):
        h = self.handle(dattn, max_context)
        cache = self.upload(dattn)
        out = torch.full((len(self.lens), self.Hq, self.D), float("nan"), device="cuda")
        h.decode(0, cache, dev(self.q), dev(self.k_new), dev(self.v_new), dev(self.pos), out,
                 gate=None if self.gate is None else dev(self.gate), write_back=write, **kw)
        assert h.get_error() == dattn.OK
        want, tol, pool = self.expect(oracle, write)
        got = out.cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        worst = (np.abs(got - want) / tol).max()
        assert worst <= 1, f"output off by {worst:.2f} of its tolerance"
        self.same_pools(pool)
        h.close()
        return got

    def same_pools(self, pool):
        for s in "kv":
            d = self.dev[s].cpu().numpy() != pool[s]
            assert not d.any(), f"{s} pool: {d.sum()} bytes differ, first at {np.argwhere(d)[0]}"


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,P,lens,rope,gate", [
    (8, 2, 256, 16, [0, 1, 15, 16, 17, 1000, 3000], (64, 5e6), True),
    (16, 8, 128, 64, [64, 200, 1, 4096], (128, 1e6), False),
    (24, 4, 256, 16, [5, 700, 33, 0], (64, 5e6), True),
    (8, 1, 128, 48, [0, 47, 48, 49, 2000], (0, 0.0), False),
    (4, 4, 128, 32, [31, 100, 32], (32, 1e4), True),
    (5, 1, 256, 16, [300, 16], (256, 1e4), False),
    (7, 1, 128, 128, [127, 500], (20, 1e4), False),
    (2, 1, 256, 80, [81, 79], (0, 0.0), True),
])
def test_decode(dattn, oracle, Hq, Hkv, D, P, lens, rope, gate, write):
    """Head layouts, pages that end inside a tile, lengths from none on."""
    Case(10 + Hq + D + P, Hq, Hkv, D, P, lens, rope, gate).check(dattn, oracle, write)


def test_decode_of_many_units(dattn, oracle):
    """As many (stream, KV head) units as a call takes, ragged, some empty."""
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 60, 64)]
    Case(20, 16, 8, 128, 16, lens, (128, 1e6)).check(dattn, oracle)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 256), (6, 1, 256), (2, 1, 128), (8, 1, 128)])
def test_decode_of_one_long_stream(dattn, oracle, Hq, Hkv, D):
    """One stream over every SM, merged across CTAs in two levels."""
    Case(30 + Hq, Hq, Hkv, D, 64, [12001], (64, 5e6)).check(dattn, oracle)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 256), (6, 1, 256), (4, 2, 128), (8, 1, 128)])
@pytest.mark.parametrize("lens", [[40], [1], [0], [700, 3], [300, 0, 17, 0, 0, 2000, 16]])
def test_decode_far_below_the_bound(dattn, oracle, Hq, Hkv, D, lens):
    """A grid for a bound of 100,000 tokens: most warps and CTAs have no block, a unit's CTAs lie far apart."""
    Case(35 + len(lens), Hq, Hkv, D, 32, lens, (64, 5e6), True).check(dattn, oracle, max_context=100000)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (16, 2, 128), (8, 4, 256), (12, 2, 256)])
def test_decode_of_tiny_units_beside_a_long_one(dattn, oracle, Hq, Hkv, D):
    """More units than warps in a CTA, whole units and parts of units in one warp's range, and a unit over many CTAs."""
    rng = np.random.default_rng(36)
    lens = [int(x) for x in rng.integers(0, 20, 40)] + [9000] + [int(x) for x in rng.integers(0, 50, 20)] + [0, 333]
    Case(37, Hq, Hkv, D, 16, lens, (32, 1e4)).check(dattn, oracle)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 96, 128, 129, 511, 512, 513, 1023, 1025])
def test_decode_around_block_borders(dattn, oracle, n):
    """Every tail of a stage of two blocks and of a window of 32."""
    Case(38, 4, 1, 128, 16, [n]).check(dattn, oracle)
    Case(39, 6, 1, 256, 32, [n]).check(dattn, oracle)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 256), (6, 1, 256), (8, 4, 128), (8, 1, 128)])
@pytest.mark.parametrize("q_mul", [8.0, 64.0, 2.0 ** -40, 0.0])
def test_decode_of_peaked_flat_and_zero_queries(dattn, oracle, Hq, Hkv, D, q_mul):
    Case(40, Hq, Hkv, D, 16, [700, 33], q_mul=q_mul).check(dattn, oracle)


def test_decode_with_qk_norm(dattn, oracle):
    Case(50, 8, 2, 256, 16, [0, 77, 500], (64, 5e6), True, norm=True).check(dattn, oracle)
    Case(51, 12, 2, 256, 16, [0, 77, 500], (256, 5e6), False, norm=True).check(dattn, oracle)


def uneven(rng, n, H, D):
    """Entries whose size grows and falls by many powers of two along the stream and between the groups."""
    x = rng.standard_normal((n, H, D)) * 2.0 ** rng.integers(-9, 9, (n, 1, 1)) * 2.0 ** rng.integers(-3, 3, (1, 1, D // 64)).repeat(64, -1)
    x[n // 2:] *= 2.0 ** -20
    x[3 * n // 4:] *= 2.0 ** 30
    return ref.bf16_bits(x)


def flat(rng, n, H, D):
    """Groups of one value, of zeros, and of two values."""
    x = rng.standard_normal((n, H, D // 64, 1)).repeat(64, -1)
    x[::3] = 0
    x[1::5, :, :, 7] = 1
    return ref.bf16_bits(x.reshape(n, H, D))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 256), (6, 1, 256), (8, 4, 128), (8, 1, 128)])
@pytest.mark.parametrize("make", [uneven, flat])
def test_decode_of_uneven_and_flat_entries(dattn, oracle, Hq, Hkv, D, make):
    Case(60, Hq, Hkv, D, 16, [900, 40], make=make, q_mul=2.0 ** -48 if make is uneven else 1.0).check(dattn, oracle)


def test_decode_of_rising_scores(dattn, oracle):
    """Every key scores higher than the one before: the running maximum moves all the time, in small and large steps."""
    def rising(rng, n, H, D):
        x = np.zeros((n, H, D))
        x[..., :] = np.sign(np.random.default_rng(70).standard_normal((1, 1, D)))
        return ref.bf16_bits(x * np.linspace(0.01, 12, n)[:, None, None] + 0.1 * rng.standard_normal((n, H, D)))
    for Hq, Hkv, D in ((8, 2, 256), (8, 1, 128)):
        c = Case(71, Hq, Hkv, D, 16, [1500, 200], make=rising)
        c.q = ref.bf16_bits(np.broadcast_to(np.sign(np.random.default_rng(70).standard_normal(D)), c.q.shape))
        c.check(dattn, oracle)


def test_a_group_without_numbers_poisons_its_head_alone(dattn, oracle):
    c = Case(80, 8, 2, 128, 16, [50, 50])
    code, lo, st = ref.load(c.pool["v"], "v", c.bt[0, 1], 3, 128)
    lo = lo.copy()
    lo[1, 0] = 0x7fc0
    ref.store(c.pool["v"], "v", c.bt[0, 1], 3, code, lo, st)
    h, cache = c.handle(dattn), c.upload(dattn)
    out = torch.zeros(2, 8, 128, device="cuda")
    h.decode(0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out)
    assert h.get_error() == dattn.OK
    nan = out.isnan().cpu().numpy()
    assert nan[0, 4:, :64].all() and not nan[0, 4:, 64:].any() and not nan[0, :4].any() and not nan[1].any()
    c.v_new[0, 0, 5] = 0x7f80  # an infinity among the new values: that group of the entry is NaN
    c.upload(dattn)
    cache = dattn.paged_cache(c.dev["k"], c.dev["v"], *c.keep)
    h.decode(0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out)
    nan = out.isnan().cpu().numpy()
    assert nan[0, :4, :64].all() and not nan[0, :4, 64:].any()
    k = torch.zeros(2, 1, 2, 128, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    h.read_kv(0, cache, c.keep[1], torch.ones_like(c.keep[1]), k, v)
    assert h.get_error() == dattn.OK
    assert v[0, 0, 0, :64].isnan().all() and not v[0, 0, 0, 64:].isnan().any() and not v[1].isnan().any()


@pytest.mark.parametrize("bad", [16 * 45 + 1, -3])
def test_a_length_outside_the_bound(dattn, oracle, bad):
    c = Case(90, 8, 2, 128, 16, [16 * 40 + 3, 16 * 45 + 30, 77])
    h, cache = c.handle(dattn, max_context=16 * 60), c.upload(dattn)
    c.keep[1][1] = bad
    out = torch.zeros(3, 8, 128, device="cuda")
    h.decode(0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out, max_seq_len=16 * 45)
    assert h.get_error() == dattn.ELENGTH
    pool = c.expect(oracle, True)[2]
    before = c.pool
    for s in "kv":  # streams 0 and 2 are written, stream 1 is not
        for b, n in ((1, 16 * 45 + 30),):
            at = c.bt[b, n // 16]
            pool[s][at] = before[s][at]
    c.same_pools(pool)


def test_steps_on_one_cache_behind_one_another(dattn, oracle):
    """Calls without a wait between them, each over what the one before it wrote, on one stream."""
    c = Case(94, 8, 2, 256, 16, [30, 200], (64, 5e6), room=20)
    h, cache = c.handle(dattn, max_context=260), c.upload(dattn)
    seq, steps, ins = c.keep[1], 18, []
    for _ in range(steps):
        q, k, v = ref.bf16_bits(c.rng.standard_normal(c.q.shape)), entries(c.rng, 2, 2, 256), entries(c.rng, 2, 2, 256)
        ins.append((q, k, v, [dev(x) for x in (q, k, v)], torch.zeros(2, 8, 256, device="cuda"),
                    seq + len(ins)))
    torch.cuda.synchronize()
    for _, _, _, d, out, pos in ins:  # (each call its own lengths, ready before the first)
        h.decode(0, dattn.paged_cache(c.dev["k"], c.dev["v"], c.keep[0], pos), *d, pos, out)
    assert h.get_error() == dattn.OK
    for i, (q, k, v, _, out, _) in enumerate(ins):
        c.q, c.k_new, c.v_new, c.pos = q, k, v, np.array(c.lens, np.int32)
        want, tol, c.pool = c.expect(oracle, True)
        assert (np.abs(out.cpu().numpy() - want) <= tol).all(), i
        for b in range(2):
            for s, e in zip("kv", c.new(oracle, b)):
                c.values[s][b] = np.concatenate([c.values[s][b], ref.value(*e)[None]])
            c.lens[b] += 1
    c.same_pools(c.pool)


def test_a_page_outside_the_pool(dattn):
    c = Case(91, 8, 2, 256, 16, [100, 100])
    h, cache = c.handle(dattn), c.upload(dattn)
    c.keep[0][1, 2] = c.pages + 7
    out = torch.zeros(2, 8, 256, device="cuda")
    h.decode(0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out, write_back=False)
    assert h.get_error() == dattn.EINDEX and h.get_error() == dattn.OK


def test_a_wait_that_runs_out(dattn, oracle):
    c = Case(92, 4, 1, 128, 16, [200])
    h, cache = c.handle(dattn), c.upload(dattn)
    out = torch.zeros(1, 4, 128, device="cuda")
    args = (0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out)
    h.debug_config(dattn.DEBUG_WITHHOLD_Q, wait_limit_us=200)
    h.decode(*args, write_back=False)
    assert h.get_error() == dattn.ETIMEOUT
    h.debug_config(0, 0)
    h.decode(*args, write_back=False)
    assert h.get_error() == dattn.OK
    want, tol, _ = c.expect(oracle, False)
    assert (np.abs(out.cpu().numpy() - want) <= tol).all()


def test_a_pool_past_32_bits(dattn, oracle):
    """Pages behind the first 4 GB of each pool."""
    c = Case(93, 8, 2, 256, 64, [200, 70], (64, 5e6), room=64)
    size = 64 // 16 * 9 * 256 * 2
    far = (1 << 32) // size + 5
    want, tol, pool = c.expect(oracle, True)
    big = {s: torch.empty(far + c.pages, *c.pool[s].shape[1:], dtype=torch.uint8, device="cuda") for s in "kv"}
    for s in "kv":
        big[s][far:] = dev(c.pool[s])
    bt = dev(np.where(c.bt >= 0, c.bt + far, -1).astype(np.int32))
    n = dev(np.array(c.lens, np.int32))
    cache = dattn.paged_cache(big["k"], big["v"], bt, n)
    h = c.handle(dattn, max_context=300)
    out = torch.zeros(2, 8, 256, device="cuda")
    h.decode(0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out)
    assert h.get_error() == dattn.OK
    assert (np.abs(out.cpu().numpy() - want) <= tol).all()
    c.dev = {s: big[s][far:] for s in "kv"}
    c.same_pools(pool)
    # and the same entries appended and read back there
    k, v = dev(c.k_new)[:, None].contiguous(), dev(c.v_new)[:, None].contiguous()
    h.append_kv(0, cache, k, v, n, torch.ones_like(n), start_pos=dev(c.pos))
    c.same_pools(pool)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    h.read_kv(0, cache, n, torch.ones_like(n), ko, vo)
    assert h.get_error() == dattn.OK
    for b in range(2):
        nk, nv = c.new(oracle, b)
        assert np.array_equal(host_u16(ko)[b, 0], ref.bf16_bits(ref.value(*nk)))
        assert np.array_equal(host_u16(vo)[b, 0], ref.bf16_bits(ref.value(*nv)))


# ---------------------------------------------------------------- append and read back

@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("D,Hkv,P,r,theta", [(256, 2, 16, 64, 5e6), (128, 8, 16, 128, 1e6), (256, 1, 64, 256, 1e4),
                                             (128, 3, 48, 20, 1e4), (128, 5, 32, 0, 0.0)])
def test_append_and_read_back(dattn, oracle, rotate, norm, D, Hkv, P, r, theta):
    """Starts inside a block, at its border and one past it; runs over several pages; rows without tokens.
    Every byte of the pools, then the entries as bf16, rows past the count left alone."""
    T = 2 * P + 21
    starts, count = [0, P - 1, P, 16 + 1, 5, 31], [T, P + 3, 1, 0, 11, 2]
    c = Case(100 + D + Hkv + P, Hkv, Hkv, D, P, [0] * 6, (r, theta), norm=norm, room=4 * P + 21)
    c.lens = starts
    rng, B = c.rng, 6
    k, v = entries(rng, B, T, Hkv, D), entries(rng, B, T, Hkv, D)
    pos = np.array([0, P - 1, 4096, 17, 300000, 9], np.int32)
    h, cache = c.handle(dattn, max_context=6 * P), c.upload(dattn)
    sd, cd = dev(np.array(starts, np.int32)), dev(np.array(count, np.int32))
    h.append_kv(0, cache, dev(k), dev(v), sd, cd, start_pos=dev(pos), rotate=rotate)
    assert h.get_error() == dattn.OK
    pool = {s: c.pool[s].copy() for s in "kv"}
    ko, vo = np.full((B, T, Hkv, D), 0x1234, np.uint16), np.full((B, T, Hkv, D), 0x1234, np.uint16)
    for b in range(B):
        for t in range(count[b]):
            at = c.bt[b, (starts[b] + t) // P], (starts[b] + t) % P
            x = np.stack([c.entry(oracle, k[b, t, j], pos[b] + t, rotate) for j in range(Hkv)])
            for s, y, o in (("k", x, ko), ("v", v[b, t], vo)):
                q = ref.quantise(ref.f64(y))
                ref.store(pool[s], s, *at, *q)
                o[b, t] = ref.bf16_bits(ref.value(*q))
    c.same_pools(pool)
    kd, vd = (torch.full((B, T, Hkv, D), 0x1234, dtype=torch.int16, device="cuda").view(torch.bfloat16) for _ in range(2))
    h.read_kv(0, cache, sd, cd, kd, vd)
    assert h.get_error() == dattn.OK
    assert np.array_equal(host_u16(kd), ko) and np.array_equal(host_u16(vd), vo)
    c.same_pools(pool)


@pytest.mark.parametrize("D", [128, 256])
def test_append_of_special_entries(dattn, D):
    """Groups with NaN, infinities, one value, tiny and huge ranges, ties: bit for bit."""
    rng = np.random.default_rng(110)
    T, H = 64, 2
    x = rng.standard_normal((1, T, H, D))
    x[0, 0:8] *= 2.0 ** rng.integers(-120, 120, (8, 1, 1))
    x[0, 8:16] = rng.integers(-30, 30, (8, H, D)) / 2
    x[0, 16:20] = 2.5
    x[0, 20:24] *= 2.0 ** -110
    x[0, 24] = 3e38 * np.sign(x[0, 24])
    x[0, 30:40] = x[0, 30:40] * 0.01 + 3
    bits = ref.bf16_bits(x)
    bits[0, 26, 0, 70], bits[0, 27, 1, 3], bits[0, 28, 0, 64] = 0x7fc0, 0x7f80, 0xff80
    c = Case(111, H, H, D, 16, [0], room=T + 1)
    h, cache = c.handle(dattn, max_context=T), c.upload(dattn)
    zero, n = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), T, dtype=torch.int32, device="cuda")
    h.append_kv(0, cache, dev(bits), dev(bits), zero, n, rotate=False)
    assert h.get_error() == dattn.OK
    pool = {s: c.pool[s].copy() for s in "kv"}
    for t in range(T):
        for s in "kv":
            ref.store(pool[s], s, c.bt[0, t // 16], t % 16, *ref.quantise(ref.f64(bits[0, t])))
    c.same_pools(pool)


@pytest.mark.parametrize("D,r", [(128, 128), (128, 64), (256, 256), (256, 40)])
def test_turned_keys_are_those_of_64_bits(dattn, D, r):
    """Keys of every size, of halves that cancel, with NaN and infinities, and dims beside the middle between two bf16 values,
    turned and stored by an append and, one stream a token, by a decode's write-back: the same bytes from both."""
    rng = np.random.default_rng(112 + D + r)
    T, H, P, theta = 64, 2, 16, 1e4
    x = rng.standard_normal((1, T, H, D))
    x[0, 0:16] *= 2.0 ** rng.integers(-126, 126, (16, 1, 1))
    x[0, 16:24] *= 2.0 ** rng.integers(-40, 40, (8, H, D))
    x[0, 24] = 3.3e38 * np.sign(x[0, 24])
    x[0, 25] = 2.0 ** -130 * np.sign(x[0, 25])
    c = Case(113, H, H, D, P, [0] * T, (r, theta), room=1)
    pos = 5 + np.arange(T)
    i = np.arange(r // 2)
    angle = pos[:, None] * theta ** (-2.0 * i / r)
    # x c = y s nearly
    t = slice(32, 48)
    x[0, t, :, :r // 2] = (x[0, t, :, r // 2:r] * np.tan(angle[t])[:, None]).clip(-1e30, 1e30)
    # x c - y s near a middle: y of that size, rounded to bf16 as it is
    t = slice(48, 64)
    mid = (1 + (2 * rng.integers(0, 128, (16, H, r // 2)) + 1) / 256) * 2.0 ** rng.integers(-3, 4, (16, H, r // 2))
    x[0, t, :, r // 2:r] = ((ref.f64(ref.bf16_bits(x[0, t, :, :r // 2])) * np.cos(angle[t])[:, None] - mid)
                            / np.sin(angle[t])[:, None]).clip(-1e30, 1e30)
    bits = ref.bf16_bits(x)
    bits[0, 26, 0, 1], bits[0, 27, 1, r - 1], bits[0, 28, 0, 3] = 0x7fc0, 0x7f80, 0xff80
    n, at = torch.full((1,), T, dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda")
    zero, h, cache = torch.zeros(1, dtype=torch.int32, device="cuda"), c.handle(dattn, max_context=T), c.upload(dattn)
    flat = Case(114, H, H, D, P, [0], (r, theta), room=T)
    hf, fc = flat.handle(dattn, max_context=T), flat.upload(dattn)
    hf.append_kv(0, fc, dev(bits), dev(bits), zero, n, start_pos=at)
    assert hf.get_error() == dattn.OK
    kv = dev(bits[0])
    h.decode(0, cache, kv, kv, kv, dev(pos.astype(np.int32)), torch.zeros(T, H, D, device="cuda"))
    assert h.get_error() == dattn.OK
    pool, fpool = ({s: y.pool[s].copy() for s in "kv"} for y in (c, flat))
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(T):
            key = ref.bf16_bits(ref.rotate(ref.f64(bits[0, t]), r, theta, int(pos[t])))
            for s, y in (("k", key), ("v", bits[0, t])):
                q = ref.quantise(ref.f64(y))
                ref.store(fpool[s], s, flat.bt[0, t // P], t % P, *q)
                ref.store(pool[s], s, c.bt[t, 0], 0, *q)
    flat.same_pools(fpool)
    c.same_pools(pool)


def test_append_and_read_of_bad_rows(dattn):
    """A count out of range, a start before 0, an index past the table and a page outside the pool are reported; the
    other rows are served and nothing else is touched."""
    c = Case(120, 2, 2, 128, 16, [0] * 4, room=40)
    T = 20
    k = dev(entries(c.rng, 4, T, 2, 128))
    for start, count, page in (([0, 0, 0, 0], [T, T + 1, -1, 1], None), ([0, -5, 60, 0], [3, 9, 9, 1], None),
                               ([0, 0, 0, 0], [T, T, 0, 1], (1, 0))):
        h, cache = c.handle(dattn, max_context=64), c.upload(dattn)
        if page:
            c.keep[0][page] = c.pages
        sd, cd = dev(np.array(start, np.int32)), dev(np.array(count, np.int32))
        h.append_kv(0, cache, k, k, sd, cd, rotate=False)
        assert h.get_error() == dattn.EINDEX
        pool = {s: c.pool[s].copy() for s in "kv"}
        src = host_u16(k)
        got = []
        for b in range(4):
            for t in range(count[b] if 0 <= count[b] <= T else 0):
                i = start[b] + t
                if i < 0 or i // 16 >= c.bt.shape[1] or (page == (b, i // 16)):
                    continue
                got.append((b, t))
                q = ref.quantise(ref.f64(src[b, t]))
                for s in "kv":
                    ref.store(pool[s], s, c.bt[b, i // 16], i % 16, *q)
        c.same_pools(pool)
        ko, vo = torch.zeros_like(k), torch.zeros_like(k)
        h.read_kv(0, cache, sd, cd, ko, vo)
        assert h.get_error() == dattn.EINDEX
        live = (ko != 0).any(-1).any(-1).cpu().numpy()
        assert {tuple(x) for x in np.argwhere(live)} == set(got)
        assert torch.equal((vo != 0).any(-1).any(-1).cpu(), torch.from_numpy(live))


@pytest.mark.parametrize("kind", ["paged", "ring"])
@pytest.mark.parametrize("fp8", [False, True])
def test_read_back_of_the_other_formats(dattn, kind, fp8):
    """bf16 entries as they are; E4M3 entries times their scale, rounded once from fp32."""
    gen, rng = synth.generator(130), np.random.default_rng(130)
    B, H, D, P, R, T = 4, 3, 128, 24, 37, 30
    rows, per = 9, (P if kind == "paged" else R)
    bits = synth.randn_bf16((rows, H, per, D), gen), synth.randn_bf16((rows, H, per, D), gen)
    scale = 0.3, 1.7
    layer = {"kind": dattn.CACHE_PAGED if kind == "paged" else dattn.CACHE_RING, "page_size": P, "ring_slots": R}
    if fp8:
        pools = [torch.from_numpy(ref.f64(b)).float().to(torch.float8_e4m3fn) for b in bits]
        layer.update(kv_format=dattn.KV_E4M3, k_scale=scale[0], v_scale=scale[1])
        want = [(p.float() * np.float32(s)).to(torch.bfloat16) for p, s in zip(pools, scale)]
    else:
        pools = [torch.from_numpy(b.view(np.int16)).view(torch.bfloat16) for b in bits]
        want = pools
    kd, vd = (p.cuda() for p in pools)
    start, count = [0, 20, 5, 40], [30, 7, 0, 30]
    if kind == "paged":
        bt = rng.permutation(rows)[:8].reshape(4, 2).astype(np.int32)
        bt = np.concatenate([bt, bt[:, :1]], 1)
        cache = dattn.paged_cache(kd, vd, dev(bt), torch.zeros(B, dtype=torch.int32, device="cuda"))
        place = lambda b, i: (bt[b, i // P], i % P)  # noqa: E731
    else:
        sr = rng.permutation(rows)[:B].astype(np.int32)
        z = torch.zeros(B, dtype=torch.int32, device="cuda")
        cache = dattn.ring_cache(kd, vd, z, z, dev(sr))
        place = lambda b, i: (sr[b], i % R)  # noqa: E731
    h = dattn.Handle(H, H, D, [layer], B, max_context=72)
    out = [torch.zeros(B, T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    h.read_kv(0, cache, dev(np.array(start, np.int32)), dev(np.array(count, np.int32)), *out)
    assert h.get_error() == dattn.OK
    for o, w in zip(out, want):
        e = torch.zeros(B, T, H, D, dtype=torch.bfloat16)
        for b in range(B):
            for t in range(count[b]):
                e[b, t] = w[place(b, start[b] + t)[0]][:, place(b, start[b] + t)[1]]
        assert torch.equal(o.cpu(), e)


def nearest_bf16(x):
    """bf16 bits nearest to fp64 values (normal numbers and zeros), ties to even, in one rounding."""
    b = np.asarray(x, np.float64).view(np.uint64)
    keep = np.uint64(45)  # 52 - 7 bits of the fraction
    b = (b + np.uint64(2 ** 44 - 1) + ((b >> keep) & np.uint64(1))) >> keep << keep
    return ref.bf16_bits(b.view(np.float64))


def test_read_back_of_e4m3_rounds_once(dattn):
    """Scales that put the product of an E4M3 value just beside the middle between two bf16 values, where fp32 has
    only the middle itself: the nearest bf16 to the exact product (by integers), of every finite byte."""
    D, P = 128, 16
    bits = np.arange(256, dtype=np.uint8)
    value = np.nan_to_num(torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy())
    hard = 0
    for m in (1.125, 1.375, 1.75, 1.625):
        for mid in range(1, 40, 2):
            scale = float(np.float32((1 + mid / 256) / m))
            exact = value * scale  # 4 + 24 bits: exact in 64
            want, twice = nearest_bf16(exact), ref.bf16_bits(exact)  # (by way of fp32)
            if (want == twice).all():
                continue
            hard += 1
            pools = [torch.from_numpy(np.tile(bits, 8 * D * P // 256).reshape(8, 1, P, D)).cuda() for _ in range(2)]
            layer = {"kind": dattn.CACHE_PAGED, "page_size": P, "kv_format": dattn.KV_E4M3, "k_scale": scale, "v_scale": scale}
            h = dattn.Handle(1, 1, D, [layer], 1, max_context=8 * P)
            bt, z = dev(np.arange(8, dtype=np.int32)[None]), torch.zeros(1, dtype=torch.int32, device="cuda")
            out = [torch.zeros(1, 8 * P, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            h.read_kv(0, dattn.paged_cache(*pools, bt, z), z, dev(np.array([8 * P], np.int32)), *out)
            assert h.get_error() == dattn.OK
            finite = np.tile(bits & 127 != 127, 8 * D * P // 256)
            for o in out:
                got = host_u16(o).reshape(-1)
                assert np.array_equal(got[finite], np.tile(want, 8 * D * P // 256)[finite])
    assert hard > 5


# ---------------------------------------------------------------- runs

def test_prompts_then_steps(dattn, oracle):
    """Prompts appended, then steps with write-back, each over what the ones before it stored; then the whole cache read
    back into a bf16 layer and decoded there."""
    c = Case(140, 8, 2, 128, 16, [0, 0, 0], (64, 1e6), room=60)
    B, T, steps = 3, 37, 6
    rng = c.rng
    k, v = entries(rng, B, T, 2, 128), entries(rng, B, T, 2, 128)
    count = np.array([37, 5, 16], np.int32)
    h = dattn.Handle(8, 2, 128, [c.layer(dattn), {"kind": dattn.CACHE_PAGED, "page_size": 16, "rotary_dim": 64,
                                                  "rope_theta": 1e6}], B, max_context=64)
    cache = c.upload(dattn)
    z = torch.zeros(B, dtype=torch.int32, device="cuda")
    h.append_kv(0, cache, dev(k), dev(v), z, dev(count), start_pos=z)
    c.lens = [int(n) for n in count]
    for b in range(B):
        x = np.stack([[c.entry(oracle, k[b, t, j], t) for j in range(2)] for t in range(count[b])])
        for s, y in (("k", x), ("v", v[b, :count[b]])):
            c.values[s][b] = ref.value(*ref.quantise(ref.f64(y)))
    seq = c.keep[1]
    seq.copy_(dev(count))
    for _ in range(steps):
        c.q = ref.bf16_bits(rng.standard_normal((B, 8, 128)))
        c.k_new, c.v_new = entries(rng, B, 2, 128), entries(rng, B, 2, 128)
        c.pos = np.array(c.lens, np.int32)
        out = torch.zeros(B, 8, 128, device="cuda")
        h.decode(0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out)
        assert h.get_error() == dattn.OK
        want, tol, _ = c.expect(oracle, False)
        assert (np.abs(out.cpu().numpy() - want) <= tol).all()
        for b in range(B):
            for s, q in zip("kv", c.new(oracle, b)):
                c.values[s][b] = np.concatenate([c.values[s][b], ref.value(*q)[None]])
            c.lens[b] += 1
        seq += 1
    n = dev(np.array(c.lens, np.int32))
    kb, vb = (torch.zeros(B, max(c.lens), 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    h.read_kv(0, cache, z, n, kb, vb)
    for b in range(B):
        assert np.array_equal(host_u16(kb)[b, :c.lens[b]], ref.bf16_bits(c.values["k"][b]))
        assert np.array_equal(host_u16(vb)[b, :c.lens[b]], ref.bf16_bits(c.values["v"][b]))
    wide = [torch.zeros(c.pages, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    flat16 = dattn.paged_cache(*wide, c.keep[0], n)
    h.append_kv(1, flat16, kb, vb, z, n, rotate=False)
    o16, o4 = torch.zeros(B, 8, 128, device="cuda"), torch.zeros(B, 8, 128, device="cuda")
    args = (dev(c.q), dev(c.k_new), dev(c.v_new), n)
    h.decode(1, flat16, *args, o16, write_back=False)
    h.decode(0, dattn.paged_cache(c.dev["k"], c.dev["v"], c.keep[0], n), *args, o4, write_back=False)
    assert h.get_error() == dattn.OK
    # bf16 values are off by 2^-9 of theirs, the new token by a step: of the size of the quantisation, not more
    assert (o16 - o4).abs().max() < 0.5


def test_layers_in_one_graph_and_on_two_streams(dattn, oracle):
    """Two 4-bit layers and a bf16 one behind one another in a captured step, replayed over new inputs; and two handles on
    two streams at once."""
    cs = [Case(150 + i, 8, 2, 256, 16, [300, 17, 0], (64, 5e6), room=4) for i in range(2)]
    h = dattn.Handle(8, 2, 256, [c.layer(dattn) for c in cs], 3, max_context=300)
    caches = [c.upload(dattn) for c in cs]
    ins = [[dev(x) for x in (c.q, c.k_new, c.v_new, c.pos)] for c in cs]
    outs = [torch.zeros(3, 8, 256, device="cuda") for _ in cs]

    def step():
        for i in range(2):
            h.decode(i, caches[i], *ins[i], outs[i])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for rep in range(3):
        for c, x, cache in zip(cs, ins, caches):
            c.q = ref.bf16_bits(c.rng.standard_normal(c.q.shape))
            c.k_new = entries(c.rng, *c.k_new.shape)
            x[0].copy_(dev(c.q))
            x[1].copy_(dev(c.k_new))
        g.replay()
        torch.cuda.synchronize()
        assert h.get_error() == dattn.OK
        for c, out in zip(cs, outs):
            want, tol, pool = c.expect(oracle, True)
            assert (np.abs(out.cpu().numpy() - want) <= tol).all()
            c.same_pools(pool)
    streams = [torch.cuda.Stream() for _ in cs]
    hs = [c.handle(dattn) for c in cs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            hs[i].decode(0, caches[i], *ins[i], outs[i], stream=streams[i])
    for i in range(2):
        assert hs[i].get_error(streams[i]) == dattn.OK
        want, tol, pool = cs[i].expect(oracle, True)
        assert (np.abs(outs[i].cpu().numpy() - want) <= tol).all()
        cs[i].same_pools(pool)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_entries_read_back_are_the_next_calls_input(dattn, fmt):
    """A decode whose new tokens the call just before it reads back, without a wait in between,
    eager and in a graph: the outputs of a decode with those tokens in place."""
    rng = np.random.default_rng(151)
    H, Hq, D, P, lens, steps = 2, 8, 128, 16, [70, 5, 33, 128], 12
    B = len(lens)
    bt, pages = tables(rng, lens, P)
    layers = [{"kind": dattn.CACHE_PAGED, "page_size": P, "kv_format": f}
              for f in (dattn.KV_INT4, dattn.KV_INT4 if fmt == "int4" else dattn.KV_BF16)]
    h = dattn.Handle(Hq, H, D, layers, B, max_context=256)
    seq = dev(np.array(lens, np.int32))
    src = dattn.paged_cache(dev(ref.random_pool(rng, pages, H, P, D)), dev(ref.random_pool(rng, pages, H, P, D)), dev(bt), seq)
    count, at = dev(np.array(lens, np.int32)), [dev(np.full(B, i % min(lens), np.int32)) for i in range(steps)]
    start, one = dev(np.zeros(B, np.int32)), dev(np.ones(B, np.int32))
    vals = [dev(entries(rng, B, max(lens), H, D)).view(torch.bfloat16) for _ in range(4)]
    h.append_kv(0, src, *vals[:2], start, count, rotate=False)
    shape = (pages, H, P, D)
    pools = [dattn.int4_pool(pages, H, P, D) if fmt == "int4" else torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    cache = dattn.paged_cache(*pools, dev(bt), seq)
    h.append_kv(1, cache, *vals[2:], start, count, rotate=False)
    q = dev(ref.bf16_bits(rng.standard_normal((B, Hq, D)))).view(torch.bfloat16)
    new = [torch.empty(B, 1, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = torch.zeros(steps, B, Hq, D, device="cuda")

    def run(wait):
        for i in range(steps):
            h.read_kv(0, src, at[i], one, *new)
            if wait:
                torch.cuda.synchronize()
            h.decode(1, cache, q, new[0].view(B, H, D), new[1].view(B, H, D), seq, out[i], max_seq_len=256, write_back=False)

    run(True)
    want = out.clone()
    assert not torch.equal(want[0], want[1])
    out.zero_()
    run(False)
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(False)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert h.get_error() == dattn.OK


def test_calls_that_do_not_take_a_4_bit_layer(dattn):
    c = Case(160, 8, 2, 128, 16, [20])
    h = c.handle(dattn, max_verify_rows=4, max_selected_pages=4)
    cache = c.upload(dattn)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out = torch.zeros(1, 8, 128, device="cuda")
    wide = torch.zeros(1, 2, 8, 128, device="cuda")
    calls = [lambda: h.verify(0, cache, x(1, 2, 8, 128), x(1, 2, 2, 128), x(1, 2, 2, 128), z.expand(1, 2).contiguous(), wide),
             lambda: h.commit(0, cache, x(1, 2, 2, 128), x(1, 2, 2, 128), z.expand(1, 2).contiguous(), z.expand(1, 2).contiguous(), z, z),
             lambda: h.prefill(0, cache, x(1, 2, 8, 128), x(1, 2, 2, 128), x(1, 2, 2, 128), z, z, wide),
             lambda: h.sparse_decode(0, cache, x(c.pages, 2, 128), x(1, 8, 128), x(1, 2, 128), x(1, 2, 128), z, out, 4),
             lambda: h.summarize(0, cache, x(c.pages, 2, 128), z, z, 1),
             lambda: dattn.decode_noalloc(h.config, 0, cache, x(1, 8, 128), x(1, 2, 128), x(1, 2, 128), z, out)]
    for call in calls:
        with pytest.raises(dattn.DattnError) as e:
            call()
        assert e.value.code == dattn.EUNSUPPORTED
    assert h.get_error() == dattn.OK
