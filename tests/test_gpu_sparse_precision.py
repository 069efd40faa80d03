"""How exact the attention over selected pages is, against 64 bits.

Bounds are relative to the softmax-weighted sum of |v| of a (head, dim), A. If
every weight p_i is off by at most e relative to itself, numerator and sum move
by e A and e, so the output by 2 e A.

Scores of keys with one dim other than zero, s (natural logarithms): q times
the scale rounds twice and q's terms (three bf16 or two fp16) drop 2^-22 at
most, the terms' sum rounds three times at 2^-24: below 2^-21 |s|. Weights add
the exponential (2^-21), P's terms (2^-22) and the sums (2^-20 for the few keys
here): e = 2^-21 |s| + 2^-19.
"""
import numpy as np
import pytest
import torch

from test_gpu_sparse import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def repeat(c, B):
    """The case's one stream B times over, in the same pages: with 304 (stream, KV head) units or more each unit is
    one CTA's, with few it is split."""
    c.lens = c.lens * B
    c.table = c.table.repeat(B, 1)
    c.pos = c.pos.repeat(B)
    c.q, c.k_new, c.v_new = c.q.repeat(B, 1, 1), c.k_new.repeat(B, 1, 1), c.v_new.repeat(B, 1, 1)
    if c.gate is not None:
        c.gate = c.gate.repeat(B, 1)
    return c


def exact(c):
    """Stream 0 over all its pages, no gate: outputs, A, and sum |q_d k_d| / sqrt(D) of the widest key of a head."""
    n = c.lens[0]
    m = -(-n // c.P)
    out, size, reach = [], [], []
    for h in range(c.Hkv):
        rows = c.table[0, :m].long()
        k = c.k.float()[rows, h].double().reshape(-1, c.D)[:n] * c.ks
        v = c.v.float()[rows, h].double().reshape(-1, c.D)[:n] * c.vs
        k1, v1 = c.entries(0, h)
        k, v = torch.cat([k, k1.double()[None] * c.ks]), torch.cat([v, v1.double()[None] * c.vs])
        q = c.rotated(0, h)
        p = torch.softmax(q @ k.T / c.D ** 0.5, -1)
        out.append(p @ v)
        size.append(p @ v.abs())
        reach.append((q.abs() @ k.abs().T).amax(-1) / c.D ** 0.5)
    return torch.cat(out), torch.cat(size), torch.cat(reach)


def check(got, want, bound):
    assert torch.isfinite(got).all()
    assert all(torch.equal(x, got[0]) for x in got)
    d = (got[0].double() - want).abs() - bound
    assert (d <= 0).all(), f"{d.max():.3g} over a bound of {bound.flatten()[d.argmax()]:.3g}"


@pytest.mark.parametrize("B", [1, 40])
def test_e4m3_many_small_weights(dattn, B):
    """Four keys without a value (one for each warp of an unsplit unit) and 4,092 keys 15 to 18 nats below them: their
    weights, 2^-22 to 2^-26, are what the output is made of. Two fp16 terms of such a weight times 2^15 leave 2^-25
    of at least 2^-11, 2^-14 in all; the scores (30 nats) add 2^-16 and the sums over 1,024 keys a warp (64 steps of
    17 addends at 2^-23, of positive values) 2^-13. e = 2^-12."""
    c = Case(31, 16, 8, 256, 16, [4096], fp8=True, r=0, gate=False)
    c.ks = 1.0
    c.q[:] = 0
    c.q[..., 0] = 16.0  # the score of a key is its dim 0
    k = torch.zeros(c.k.shape)
    k[..., 0] = torch.randint(12, 16, c.k.shape[:3], generator=c.g).float()
    v = torch.rand(c.v.shape, generator=c.g) + 0.5
    first = c.table[0, :4].long()
    k[first, :, 0, 0] = 30.0
    v[first, :, 0] = 0.0
    c.k, c.v = k.to(c.kind), v.to(c.kind)
    c.k_new[:] = 0
    want, size, _ = exact(c)
    out, _ = repeat(c, B).run(dattn, 300, 1, 1)
    check(out, want, 2 * 2.0 ** -12 * size)


@pytest.mark.parametrize("fp8", [False, True])
def test_heads_of_very_different_sizes(dattn, fp8):
    """One query head of a group 2^12 times the others: theirs keep their own precision."""
    c = Case(32, 8, 2, 128, 16, [100], fp8=fp8, r=0, gate=False)
    c.ks = 1.0
    c.q = (100 + 28 * torch.rand(c.q.shape, generator=c.g)).to(torch.bfloat16)
    c.q[:, ::4] *= 2.0 ** 12
    one_hot(c)
    want, size, reach = exact(c)
    out, _ = c.run(dattn, 8, 1, 1)
    check(out[:, [1, 2, 3, 5, 6, 7]], want[[1, 2, 3, 5, 6, 7]],
          2 * ((reach * 2.0 ** -21 + 2.0 ** -19)[:, None] * size)[[1, 2, 3, 5, 6, 7]])


def one_hot(c, least=0):
    """Keys of one dim each, 1 in dim i for token i + least; the new token's is the last dim."""
    k = torch.zeros(c.k.shape)
    for i in range(c.lens[0]):
        k[int(c.table[0, i // c.P]), :, i % c.P, i + least] = 1.0
    c.k = k.to(c.kind)
    c.k_new[:] = 0
    c.k_new[..., c.D - 1] = 1.0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [1, 160])
def test_large_scores_keep_their_low_bits(dattn, fp8, B):
    """Scores of 35 to 44 nats from single dims: nothing but the query's terms, its scale and the sum of the terms
    stands between them and the weights. (Two bf16 terms instead of three miss by up to 2^-18 of the score.)"""
    c = Case(33, 8, 2, 128, 16, [100], fp8=fp8, r=0, gate=False)
    c.ks = 1.0
    c.q = (400 + 100 * torch.rand(c.q.shape, generator=c.g)).to(torch.bfloat16)
    one_hot(c)
    want, size, reach = exact(c)
    out, _ = repeat(c, B).run(dattn, 8, 1, 1)
    check(out, want, 2 * (reach * 2.0 ** -21 + 2.0 ** -19)[:, None] * size)


@pytest.mark.parametrize("where", [[], [0], [350], [699], [699, 350, 3], [3, 350, 699], "new"])
@pytest.mark.parametrize("q_mul", [1, 8, 32])
@pytest.mark.parametrize("fp8,B", [(False, 1), (False, 160), (True, 1), (True, 160)])
def test_peaked_rows(dattn, fp8, B, q_mul, where):
    """Keys along the group's query at the beginning, in the middle and at the end, each one larger than the one before
    it in the list (the running maximum jumps, or is there at once), or the new token's.

    Scores: an MMA adds 16 products to its sum, each of the 17 off by 2^-23 of the largest at most, 4 MMAs a chain at D
    = 128, and the query's rounding: (4 * 17 * 2^-23 + 2^-20) sum |q_d k_d| / sqrt(D) nats. Outputs: 11 groups a warp of
    three terms each, 17 * 2^-23 an MMA.

    Where the keys with weight have no value in a dim, A is next to nothing and what small weights lose shows: a weight
    below 2^-126 of its warp's largest is 0, and E4M3's terms of 2^15 p end at 2^-24, so that each of the 701 weights
    is off by 2^-25 2^-15 = 2^-40 of a sum of at least 1 (after the joins: of more)."""
    c = Case(34, 8, 2, 128, 16, [700], fp8=fp8, r=0, gate=False, q_mul=q_mul)
    along = c.q.float().view(2, 4, 128).mean(1)
    along /= along.pow(2).mean(-1, keepdim=True).sqrt()
    if where == "new":
        c.k_new = (3 * along)[None].to(torch.bfloat16)
    else:
        k = c.k.float()
        for i, t in enumerate(where):
            k[int(c.table[0, t // 16]), :, t % 16] = (2 + i) * along
        c.k = k.to(c.kind)
    want, size, reach = exact(c)
    out, _ = repeat(c, B).run(dattn, 64, 1, 1)
    e = reach * (4 * 17 * 2.0 ** -23 + 2.0 ** -20) + 11 * 3 * 17 * 2.0 ** -23 + 2.0 ** -19
    check(out, want, 2 * e[:, None] * size + 701 * (2.0 ** -40 if fp8 else 2.0 ** -126) * c.v.float().abs().max().item() * c.vs)
