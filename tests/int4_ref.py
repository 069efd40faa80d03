"""The 4-bit cache written out in 64 bits (numpy): quantisation of an entry and the
place of its bits in a pool, from the description in include/dattn.h; and decode
attention over such a pool."""
import numpy as np

BLOCK, GROUP = 16, 64


def f64(bits):
    """bf16 bit patterns as fp64."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_bits(x):
    """Nearest bf16 (ties to even) of finite values that fp32 holds or that are not near a bf16 midpoint."""
    x = np.asarray(x, np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    return ((b + 0x7fff + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def quantise(x):
    """Entries [..., D] (fp64 of bf16 values) -> codes [..., D], least and step [..., D / 64] as bf16 bits.

    x - least is rounded to fp32, as the format says. It is a multiple of the smaller one's last bit and below twice
    the larger one, so fp32's 24 bits hold it where the two are within 2^15 of one another: then nothing is rounded."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(invalid="ignore", over="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        ok = np.isfinite(g).all(-1) & (hi - lo <= 3.402823466e38)
        lo, width = np.where(ok, lo, 0.0), np.where(ok, hi - lo, 0.0)
    sb = bf16_bits(width / 15)
    step = f64(sb)
    step = np.where(step < 2.0 ** -100, 0.0, step)
    lb = np.where(ok, bf16_bits(lo), 0x7fc0).astype(np.uint16)
    sb = np.where(step == 0, 0, sb).astype(np.uint16)
    d = np.where(ok[..., None], np.float32(np.where(ok[..., None], g - lo[..., None], 0.0)).astype(np.float64), 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(step[..., None] > 0, np.rint(d / step[..., None]), 0.0)
    return code.clip(0, 15).astype(np.uint8).reshape(x.shape), lb, sb


def value(code, least, step):
    """What codes stand for."""
    g = code.reshape(*code.shape[:-1], code.shape[-1] // GROUP, GROUP).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return (f64(least)[..., None] + g * f64(step)[..., None]).reshape(code.shape)


def code_byte(side, D, r, d):
    """Byte of a block that holds the code of dim d of token r (even dims in its low half)."""
    r, d = np.asarray(r), np.asarray(d)
    if side == "k":
        return d // 128 * 1024 + r * 64 + d // 16 % 4 * 16 + d // 64 % 2 * 8 + d % 16 // 2
    return d // 64 * 512 + (d // 8 % 8 * 4 + r % 8 // 2) * 16 + r // 8 * 8 + d // 4 % 2 * 4 + r % 2 * 2 + d % 4 // 2


def pair_byte(D, r, G):
    return 8 * D + (np.asarray(r) * (D // GROUP) + np.asarray(G)) * 4


def store(pool, side, page, at, code, least, step):
    """One token's entries of every head ([H, D], [H, D / 64]) at place `at` of a page of pool [pages, H, bytes]."""
    H, D = code.shape
    blk, r = (at // BLOCK) * 9 * D, at % BLOCK
    even = np.arange(0, D, 2)
    b = blk + code_byte(side, D, r, even)
    pool[page][:, b] = code[:, even] | (code[:, even + 1] << 4)
    for G in range(D // GROUP):
        p = blk + int(pair_byte(D, r, G))
        pool[page, :, p:p + 2] = np.ascontiguousarray(least[:, G:G + 1]).view(np.uint8)
        pool[page, :, p + 2:p + 4] = np.ascontiguousarray(step[:, G:G + 1]).view(np.uint8)


def load(pool, side, page, at, D):
    """One token's codes and pairs of every head."""
    blk, r = (at // BLOCK) * 9 * D, at % BLOCK
    d = np.arange(D)
    code = (pool[page][:, blk + code_byte(side, D, r, d)] >> (d % 2 * 4)) & 15
    p = blk + int(pair_byte(D, r, 0))
    pairs = np.ascontiguousarray(pool[page, :, p:p + D // GROUP * 4]).view(np.uint16).reshape(-1, D // GROUP, 2)
    return code, pairs[..., 0], pairs[..., 1]


def random_pool(rng, pages, H, P, D):
    """A pool of bytes that are no entry: every least value and step is a NaN."""
    pool = rng.integers(0, 256, (pages, H, P // BLOCK, 9 * D), dtype=np.uint8)
    pool[..., 8 * D:] = 0xff
    return pool.reshape(pages, H, P // BLOCK * 9 * D)


def attend(q, k, v, scale, gate=None):
    """One stream and KV head: q [G, D], k, v [n, D] fp64 -> [G, D]; gate [G]."""
    s = (q @ k.T) * scale
    a = np.exp(s - s.max(-1, keepdims=True))
    o = (a / a.sum(-1, keepdims=True)) @ v
    return o if gate is None else o / (1 + np.exp(-gate))[:, None]


def rotate(x, r, theta, pos):
    """[.., D] fp64 turned at pos in pairs (i, i + r / 2)."""
    if r == 0:
        return x
    i = np.arange(r // 2)
    a = pos * theta ** (-2.0 * i / r)
    c, s = np.cos(a), np.sin(a)
    y = x.copy()
    y[..., :r // 2] = x[..., :r // 2] * c - x[..., r // 2:r] * s
    y[..., r // 2:r] = x[..., r // 2:r] * c + x[..., :r // 2] * s
    return y
