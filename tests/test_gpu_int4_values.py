"""Decode over 4-bit caches whose values differ by many powers of two: what a huge value that
a head gives no weight leaves of the others.

Tolerance of one output, from the 64-bit softmax p and A_k, the largest value of key k in the
output's group of 64 dims (what its grid's parts are of the size of): a score is off by
e_k = (2^-22 + 4 sqrt(D) 2^-24) |q| . |k| / sqrt(D) at the most - q as two fp16 terms, fp32
sums of D products taken as four times their walk of D roundings -, which moves an output by
sum p_k e_k (A_k + A), A = sum p_k A_k; the weights' two fp16 terms (2^-22 of them, or 2^-30 of
the largest product of weight and step that their warp has met: for its 64 keys 2^-24 of what A
has of them) and the fp32 sums are within 2^-20 A.
"""
import numpy as np
import pytest
import torch

import int4_ref as ref
from gpu_util import dev
from test_gpu_int4 import Case, dattn  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def expect(c, b):
    """Outputs and tolerances of stream b: [Hq, D] both."""
    G, D = c.Hq // c.Hkv, c.D
    out, tol = np.empty((c.Hq, D)), np.empty((c.Hq, D))
    nk, nv = c.new(None, b)
    for j in range(c.Hkv):
        k = np.concatenate([c.values["k"][b][:, j], ref.value(*nk)[j:j + 1]])
        v = np.concatenate([c.values["v"][b][:, j], ref.value(*nv)[j:j + 1]])
        A = np.abs(v).reshape(len(v), -1, 64).max(-1).repeat(64, -1)
        for i in range(j * G, (j + 1) * G):
            q = ref.f64(c.q[b, i])
            s = k @ q * D ** -0.5
            p = np.exp(s - s.max())
            p /= p.sum()
            e = (2.0 ** -22 + 4 * D ** 0.5 * 2.0 ** -24) * (np.abs(k) @ np.abs(q)) * D ** -0.5
            out[i] = p @ v
            tol[i] = (p * e) @ A + ((p * e).sum() + 2.0 ** -20) * (p @ A)
    return out, tol


def run(dattn, c):
    h, cache = c.handle(dattn), c.upload(dattn)
    out = torch.full((len(c.lens), c.Hq, c.D), float("nan"), device="cuda")
    h.decode(0, cache, dev(c.q), dev(c.k_new), dev(c.v_new), dev(c.pos), out, write_back=False)
    assert h.get_error() == dattn.OK
    got = out.cpu().numpy().astype(np.float64)
    for b in range(len(c.lens)):
        want, tol = expect(c, b)
        off = np.abs(got[b] - want) / tol
        assert off.max() <= 1, f"stream {b}: output {np.unravel_index(off.argmax(), off.shape)} off by {off.max():.3g} of its tolerance"


def sides(D):
    return np.sign(np.random.default_rng(7).standard_normal(D))


def with_huge(at, size):
    """Keys and values of size 1, but for the token `at`: its key is 5 on the sides, the values of its first group (and of
    the last, negative) are of that size."""
    def make(rng, n, H, D):
        x = rng.standard_normal((n, H, D)) * 0.5
        if make.calls % 2 == 0:
            x[at] = 5 * sides(D)
        else:
            x[at, :, :64] *= size
            x[at, :, -64:] *= -size
        make.calls += 1
        return ref.bf16_bits(x)
    make.calls = 0
    return make


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 256), (6, 1, 256), (4, 2, 128), (8, 1, 128)])
@pytest.mark.parametrize("at", [0, 700, 1500])
@pytest.mark.parametrize("bits", [16, 24, 40, 70])
def test_a_huge_value_without_weight(dattn, Hq, Hkv, D, at, bits):  # noqa: F811
    """Even heads give the token nothing (e^-60 and less of the others), odd ones nearly everything: neither may cost the
    other its weights' bits."""
    c = Case(300 + bits + at + Hq + D, Hq, Hkv, D, 16, [1600], make=with_huge(at, 2.0 ** bits))
    c.k_new = ref.bf16_bits(c.rng.standard_normal(c.k_new.shape) * 0.5)
    lean = np.where(np.arange(Hq) % 2 == 0, -1.5, 1.0)[:, None] * sides(D) * (60 / 57) * (256 / D) ** 0.5
    c.q = ref.bf16_bits(c.rng.standard_normal((1, Hq, D)) * 0.5 + lean)
    run(dattn, c)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 256), (6, 1, 256), (4, 2, 128), (8, 1, 128)])
def test_values_that_fall_and_rise_with_their_scores(dattn, Hq, Hkv, D):  # noqa: F811
    """Along the stream scores rise by 80 and values fall by 2^60, then the other way round; and groups that do neither."""
    def make(rng, n, H, D):
        x = rng.standard_normal((n, H, D)) * 0.3
        t = np.abs(np.linspace(-1, 1, n))[:, None]  # 1 .. 0 .. 1
        if make.calls % 2 == 0:
            x += (5 * (1 - t) * sides(D))[:, None]
        else:
            x[:, :, :64] *= 2.0 ** np.rint(60 * t)[:, None]
        make.calls += 1
        return ref.bf16_bits(x)
    make.calls = 0
    c = Case(400 + Hq + D, Hq, Hkv, D, 16, [1500], make=make)
    c.k_new = ref.bf16_bits(c.rng.standard_normal(c.k_new.shape) * 0.3 + 2 * sides(D))
    c.q = ref.bf16_bits(c.rng.standard_normal((1, Hq, D)) * 0.3 + np.linspace(0.3, 1.2, Hq)[:, None] * sides(D) * (256 / D) ** 0.5)
    run(dattn, c)
