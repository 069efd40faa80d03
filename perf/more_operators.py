"""Measured cases of the 4-bit cache: entries quantised as they are written, read
back as bf16, and decode attention over them.

A paged cache in 4 bits holds, for every token and KV head, D codes of 4 bits and,
for each group of 64 dims, the group's least value and its step (bf16 both): the
value of a code is least + code * step. Sixteen tokens of a head are one block of
9 D bytes: their codes in the order in which the matrix instructions take them (for
K and V each its own, see _codes), then the tokens' (least, step) pairs.

Each case is run in a plain form (elementary torch operations in 32 bits, the codes'
rounding in 64) or, with `own` set, through the library's entry points. Head layouts,
page sizes and context lengths are those of the repository's benchmark: 8 query / 2 KV
heads of 256, 16 / 8 heads of 128, 24 / 4 heads of 256; 16- and 64-token pages; up to
1,048,576 cached tokens. The keys of the decode cases carry no rotation: a rotated
entry next to the border of two codes would be one thing or the other by its last bit.
"""
import math
import random

import torch

own = False

THETA = 1e6
GROUP = 64


def listed():
    return [
        # decode of one very long stream
        {"name": "decode 1 x 1048576", "op": "decode", "streams": 1, "lo": 1048576, "hi": 1048576, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "page": 64, "gate": False, "write": False},
        # the long-context batch of the benchmark
        {"name": "decode 8 x 262144", "op": "decode", "streams": 8, "lo": 262144, "hi": 262144, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "page": 64, "gate": False, "write": False},
        # a full serving batch with ragged lengths in small pages
        {"name": "decode 64 ragged", "op": "decode", "streams": 64, "lo": 64, "hi": 4096, "q_heads": 16,
         "kv_heads": 8, "dim": 128, "page": 16, "gate": False, "write": False},
        # six query heads to a KV head, lengths near one another
        {"name": "decode 32 x 16384", "op": "decode", "streams": 32, "lo": 15000, "hi": 16384, "q_heads": 24,
         "kv_heads": 4, "dim": 256, "page": 16, "gate": True, "write": False},
        # one interactive stream, the new entry written and read back as the next step will see it: latency counts
        {"name": "decode 1 x 5003 write", "op": "decode", "streams": 1, "lo": 5003, "hi": 5003, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "page": 16, "gate": True, "write": True},
        # a batch's prompts, rotated and written, and read back as later steps will see them
        {"name": "append 64 ragged", "op": "append", "streams": 64, "lo": 64, "hi": 4096, "q_heads": 16,
         "kv_heads": 8, "dim": 128, "page": 16, "rotary": 128, "start": 0},
        # one long prompt whose keys come rotated, behind a cached one of odd length
        {"name": "append 1 x 32768", "op": "append", "streams": 1, "lo": 32768, "hi": 32768, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "page": 64, "rotary": 0, "start": 1001},
        # one token a stream
        {"name": "append step", "op": "append", "streams": 64, "lo": 1, "hi": 1, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "page": 16, "rotary": 64, "start": 500},
        # a batch's caches handed on as bf16
        {"name": "read 64 ragged", "op": "read", "streams": 64, "lo": 64, "hi": 4096, "q_heads": 16,
         "kv_heads": 8, "dim": 128, "page": 16, "start": 0},
        # a shared prefix of one stream
        {"name": "read 1 x 131072", "op": "read", "streams": 1, "lo": 131072, "hi": 131072, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "page": 64, "start": 0},
        # the last turns of a few streams
        {"name": "read 4 short", "op": "read", "streams": 4, "lo": 1, "hi": 150, "q_heads": 24,
         "kv_heads": 4, "dim": 256, "page": 16, "start": 777},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "read"])
    qh, kvh, dim = rng.choice([(8, 2, 256), (16, 8, 128), (24, 4, 256), (8, 8, 128), (6, 2, 128), (8, 1, 128), (5, 1, 256)])
    c = {"op": op, "q_heads": qh, "kv_heads": kvh, "dim": dim, "page": rng.choice([16, 16, 32, 48, 64, 128]),
         "streams": _log(rng, 1, 64)}
    if op == "decode":
        most = 524288 * 512 // (kvh * dim)
        hi = _log(rng, 16, max(17, min(262144, most // c["streams"])))
        c.update(lo=rng.choice([hi, max(1, hi // 8), 0]), hi=hi, gate=rng.random() < 0.5, write=rng.random() < 0.3)
    else:
        most = 131072 * 1024 // (kvh * dim)
        hi = _log(rng, 1, max(2, min(32768, most // c["streams"])))
        c.update(lo=rng.choice([hi, max(1, hi // 8), 0]), hi=hi, start=rng.choice([0, 16, rng.randint(1, 2000)]))
        if op == "append":
            c["rotary"] = rng.choice([dim, dim // 4, 0, 0])
    return c


def _lens(case):
    """The batch's lengths: uniform in [lo, hi], the same for every seed (the work depends on them)."""
    rng = random.Random(case["streams"] * 1000003 + case["hi"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["streams"])]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _entries(g, *shape):
    """Keys or values as a cache meets them: dims of unlike spread, some of them off zero."""
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    dim = torch.arange(shape[-1], device="cuda")
    return (x * (0.5 + (dim % 7) / 4.0) + (dim % 13 == 0) * 2.0).to(torch.bfloat16)


def _filled(g, pages, heads, page, dim, keys):
    """A pool [pages, heads, bytes] of quantised entries."""
    pool = torch.empty(pages, heads, page * dim * 9 // 16, device="cuda", dtype=torch.uint8)
    step = max(1, (1 << 26) // (heads * page * dim))
    at = torch.arange(page, device="cuda")
    for p0 in range(0, pages, step):
        n = min(step, pages - p0)
        code, least, width = _quantised(_entries(g, n, page, heads, dim))
        rows = torch.arange(p0, p0 + n, device="cuda")[:, None]
        _store(pool, keys, rows, at[None], code, least, width)
    return pool


def prepare(case, seed):
    g = _generator(seed)
    H, D, S, P = case["kv_heads"], case["dim"], case["streams"], case["page"]
    lens = _lens(case)
    s = {"case": case}
    first = case.get("start", 0)
    room = [(first + n) // P + 1 for n in lens]
    total = sum(room) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([0] + room[:-1]).cumsum(0)[:, None] + torch.arange(max(room))[None]
    inside = torch.arange(max(room))[None] < torch.tensor(room)[:, None]
    s["table"] = torch.where(inside.cuda(), perm[at.clamp(max=total - 1).cuda()], -1).to(torch.int32).contiguous()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        s["k"] = torch.zeros(total, H, P * D * 9 // 16, device="cuda", dtype=torch.uint8)
        s["v"] = torch.zeros_like(s["k"])
    else:
        s["k"], s["v"] = _filled(g, total, H, P, D, True), _filled(g, total, H, P, D, False)
    if case["op"] == "decode":
        s.update(seq=n, q=_normal(g, S, case["q_heads"], D), k_new=_entries(g, S, H, D), v_new=_entries(g, S, H, D),
                 gate=_normal(g, S, case["q_heads"]) if case["gate"] else None, pos=n.clone(),
                 out=torch.zeros(S, case["q_heads"], D, device="cuda"))
        s.update(start=n.clone(), count=torch.ones_like(n))
    else:
        s.update(start=torch.full_like(n, first), count=n, seq=n + first, pos=torch.full_like(n, first))
        if case["op"] == "append":
            s.update(k_new=_entries(g, S, case["hi"], H, D), v_new=_entries(g, S, case["hi"], H, D))
    T = 1 if case["op"] == "decode" else case["hi"]
    s["k_out"] = torch.zeros(S, T, H, D, device="cuda", dtype=torch.bfloat16)
    s["v_out"] = torch.zeros_like(s["k_out"])
    if own:
        import decode_attention_kv_dattn_gb300 as dattn
        layer = {"kind": dattn.CACHE_PAGED, "page_size": P, "rotary_dim": case.get("rotary", 0), "rope_theta": THETA,
                 "kv_format": dattn.KV_INT4}
        s["handle"] = dattn.Handle(case["q_heads"], H, D, [layer], S, max_context=first + max(max(lens), 1))
        s["cache"] = dattn.paged_cache(s["k"], s["v"], s["table"], s["seq"])
    return s


# ---------------------------------------------------------------- plain forms

def _quantised(x):
    """Codes [..., D], and the least value and the step [..., D / 64] of each group, of bf16 entries [..., D]."""
    x = x.float().unflatten(-1, (-1, GROUP))
    least, most = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    width = ((most - least) / 15).to(torch.bfloat16).float()
    width = torch.where(width < 2.0 ** -100, 0, width)
    # 64 bits: the border between two codes
    code = ((x.double() - least.double()) / torch.where(width > 0, width, 1).double()).round().clamp(0, 15)
    return code.to(torch.uint8).flatten(-2), least[..., 0].to(torch.bfloat16), width[..., 0].to(torch.bfloat16)


def _codes(pool, D, keys):
    """The codes of a pool's 16-token blocks as a view, the token's place in the block and then the order of a
    token's bytes last: [rows, heads, blocks, (token), (bytes)]. K: sections of 128 dims, each 16 tokens x 64 bytes, in
    which 16 bytes hold 16 dims of the first group and 16 of the second. V: groups of 64 dims, in which 16 bytes hold 8
    dims of tokens t, t + 1, t + 8, t + 9."""
    blocks = pool.unflatten(-1, (-1, 9 * D))[..., :8 * D]
    if keys:
        return blocks.unflatten(-1, (D // 128, 16, 4, 2, 2, 4)).permute(0, 1, 2, 4, 3, 6, 5, 7, 8)
    return blocks.unflatten(-1, (D // 64, 8, 4, 2, 2, 2, 2)).permute(0, 1, 2, 6, 5, 8, 3, 4, 7, 9)


def _pairs(pool, D):
    """The (least, step) pairs of a pool's blocks as a view: [rows, heads, blocks, token, groups, 2] bf16."""
    return pool.view(torch.bfloat16).unflatten(-1, (-1, 9 * D // 2))[..., 4 * D:].unflatten(-1, (16, D // GROUP, 2))


def _store(pool, keys, rows, at, code, least, width):
    """Entries [n, tokens, heads, D] into place `at` of pages `rows` (both [n, tokens])."""
    D = code.shape[-1]
    rows, at = torch.broadcast_tensors(rows, at)
    rows, block, t = rows[..., None], (at // 16)[..., None], (at % 16)[..., None]
    h = torch.arange(code.shape[-2], device=code.device)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    view = _codes(pool, D, keys)
    if keys:
        view[rows, h, block, t] = packed.unflatten(-1, view.shape[4:])
    else:
        view[rows, h, block, t // 8, t % 8 // 2, t % 2] = packed.unflatten(-1, view.shape[6:])
    _pairs(pool, D)[rows, h, block, t] = torch.stack([least, width], -1)


def _values(pool, D, keys, rows):
    """The values of pages `rows` [...] in 32 bits: [..., heads, tokens, D]."""
    pages = pool[rows].flatten(0, -3)
    byte = _codes(pages, D, keys)
    byte = byte.reshape(*byte.shape[:3], 16, D // 2)
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).float()
    pair = _pairs(pages, D).float()
    x = pair[..., :1] + code.unflatten(-1, (-1, GROUP)) * pair[..., 1:]
    return x.flatten(-2).flatten(2, 3).unflatten(0, rows.shape)


def _rotated(x, pos, rotary):
    """x [B, T, heads, D] bf16, the first `rotary` dims turned at pos [B, T] in pairs (i, i + rotary / 2), as bf16."""
    if not rotary:
        return x
    half = rotary // 2
    freq = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) * 2 / rotary)
    angle = pos.double()[..., None, None] * freq
    c, s = angle.cos(), angle.sin()
    a, b = x[..., :half].double(), x[..., half:rotary].double()
    return torch.cat([(a * c - b * s).to(torch.bfloat16), (b * c + a * s).to(torch.bfloat16), x[..., rotary:]], -1)


def _places(s):
    """Page and place of tokens start + t, t < T, of each stream, and which of them there are."""
    P, T = s["case"]["page"], s["k_out"].shape[1]
    t = torch.arange(T, device="cuda")
    live = t < s["count"][:, None]
    at = s["start"].long()[:, None] + torch.where(live, t, 0)
    return torch.gather(s["table"].long(), 1, (at // P).clamp(max=s["table"].shape[1] - 1)), at % P, live


def _append(s):
    rows, at, live = _places(s)
    pos = s["pos"][:, None] + torch.arange(live.shape[1], device="cuda")
    for pool, x, keys in ((s["k"], _rotated(s["k_new"], pos, s["case"]["rotary"]), True), (s["v"], s["v_new"], False)):
        code, least, width = _quantised(x[live][:, None])
        _store(pool, keys, rows[live][:, None], at[live][:, None], code, least, width)


def _read(s):
    D, P = s["case"]["dim"], s["case"]["page"]
    rows, at, live = _places(s)
    for pool, out, keys in ((s["k"], s["k_out"], True), (s["v"], s["v_out"], False)):
        x = _values(pool, D, keys, s["table"].long().clamp(min=0)).to(torch.bfloat16)  # [B, pages, heads, P, D]
        x = x.transpose(2, 3).flatten(1, 2)
        t = s["start"].long()[:, None] + torch.arange(live.shape[1], device="cuda")
        x = torch.gather(x, 1, t.clamp(max=x.shape[1] - 1)[..., None, None].expand(-1, -1, *x.shape[2:]))
        out.copy_(torch.where(live[..., None, None], x, out))
    return s["k_out"], s["v_out"]


def _decode(s):
    case = s["case"]
    B, H, D, P = case["streams"], case["kv_heads"], case["dim"], case["page"]
    G = case["q_heads"] // H
    n = s["seq"].long()
    rows = s["table"].long().clamp(min=0)
    k, v = (_values(s[x], D, x == "k", rows).transpose(1, 2).flatten(2, 3) for x in ("k", "v"))  # [B, heads, tokens, D]
    valid = torch.arange(k.shape[2], device="cuda") < n[:, None]
    new = []
    for x in (s["k_new"], s["v_new"]):
        code, least, width = _quantised(x)
        new.append((code, least, width, (least.float()[..., None] + code.float().unflatten(-1, (-1, GROUP)) *
                                         width.float()[..., None]).flatten(-2)))
    q = s["q"].float().view(B, H, G, D) / math.sqrt(D)
    a = torch.einsum("bhgd,bhnd->bhgn", q, k)
    a = torch.where(valid[:, None, None], a, -math.inf)
    a = torch.cat([a, torch.einsum("bhgd,bhd->bhg", q, new[0][3])[..., None]], -1)
    a = (a - a.amax(-1, keepdim=True)).exp()
    total = a.sum(-1, keepdim=True)
    v = torch.where(valid[:, None, :, None], v, 0)
    out = torch.einsum("bhgn,bhnd->bhgd", a[..., :-1], v) + a[..., -1:] * new[1][3][:, :, None]
    out = (out / total).reshape(B, H * G, D)
    if case["gate"]:
        out = out / (1 + (-s["gate"].float()).exp())[..., None]
    if case["write"]:
        at = torch.gather(rows, 1, (n // P)[:, None])
        _store(s["k"], True, at, (n % P)[:, None], *(x[:, None] for x in new[0][:3]))
        _store(s["v"], False, at, (n % P)[:, None], *(x[:, None] for x in new[1][:3]))
    return out


def run(s):
    case = s["case"]
    if case["op"] == "decode":
        if own:
            s["handle"].decode(0, s["cache"], s["q"], s["k_new"], s["v_new"], s["pos"], s["out"], gate=s["gate"],
                               write_back=case["write"])
            if case["write"]:
                s["handle"].read_kv(0, s["cache"], s["start"], s["count"], s["k_out"], s["v_out"])
            return (s["out"], s["k_out"], s["v_out"]) if case["write"] else s["out"]
        out = _decode(s)
        return (out, *_read_new(s)) if case["write"] else out
    if own:
        if case["op"] == "append":
            s["handle"].append_kv(0, s["cache"], s["k_new"], s["v_new"], s["start"], s["count"], start_pos=s["pos"],
                                  rotate=case["rotary"] > 0)
        s["handle"].read_kv(0, s["cache"], s["start"], s["count"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if case["op"] == "append":
        _append(s)
    return _read(s)


def _read_new(s):
    """The entry at seq of each stream as it is stored."""
    D, P = s["case"]["dim"], s["case"]["page"]
    n = s["seq"].long()
    rows = torch.gather(s["table"].long(), 1, (n // P)[:, None])
    at = (n % P)[:, None, None, None, None]
    pick = lambda x: torch.gather(x, 3, at.expand(*x.shape[:3], 1, D))[:, 0, :, 0].to(torch.bfloat16)  # noqa: E731
    s["k_out"][:, 0] = pick(_values(s["k"], D, True, rows))
    s["v_out"][:, 0] = pick(_values(s["v"], D, False, rows))
    return s["k_out"], s["v_out"]


def work(case):
    H, D, S, Q = case["kv_heads"], case["dim"], case["streams"], case["q_heads"]
    n = sum(_lens(case))
    entry = 2 * H * D * 9 // 16  # bytes of a cached token
    if case["op"] == "decode":
        io = S * ((Q + 2 * H) * D * 2 + Q * D * 4 + 12)
        if case["write"]:
            io += S * (entry + 2 * H * D * 2)
        return {"bytes": n * entry + io, "flops": n * Q * D * 4}
    # append: the entries read once, written in 4 bits and returned as bf16
    new = 2 * H * D * 2 if case["op"] == "append" else 0
    return {"bytes": n * (entry + 2 * H * D * 2 + new) + S * 12, "flops": n * 2 * H * D * (2 + (6 if new else 0))}


# ---------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    H, D, S, P, Q = case["kv_heads"], case["dim"], case["streams"], case["page"], case["q_heads"]
    d = torch.arange(D, device="cuda")
    r = torch.arange(16, device="cuda")[:, None]
    # where the code of dim d of token r of a block is (byte), and where its group's pair is (bf16)
    where = {"k": d // 128 * 1024 + r * 64 + d % 64 // 16 * 16 + d % 128 // 64 * 8 + d % 16 // 2,
             "v": d // 64 * 512 + (d % 64 // 8 * 4 + r % 8 // 2) * 16 + r // 8 * 8 + d % 8 // 4 * 4 + r % 2 * 2 + d % 4 // 2}
    pair = 4 * D + (r * (D // 64) + d // 64) * 2

    def values(which, rows):
        """[heads, tokens, D] of the pages `rows` of a stream."""
        blocks = s[which][rows].view(len(rows), H, P // 16, 9 * D)
        code = (blocks[..., where[which]].int() >> (d % 2 * 4)) & 15
        b16 = blocks.view(torch.bfloat16)
        x = b16[..., pair].double() + code * b16[..., pair + 1].double()
        return x.permute(1, 0, 2, 3, 4).reshape(H, len(rows) * P, D)

    def stored(x):
        """Entries as the cache holds them: [..., D] to their values."""
        x = x.double().view(*x.shape[:-1], D // 64, 64)
        lo = x.min(-1, keepdim=True).values
        step = ((x.max(-1, keepdim=True).values - lo) / 15).to(torch.bfloat16).double()
        step[step < 2.0 ** -100] = 0
        code = torch.where(step == 0, step, torch.round((x - lo) / step)).clamp(0, 15)
        return (lo + step * code).view(*x.shape[:-2], D)

    if case["op"] == "decode":
        out = torch.empty(S, Q, D, device="cuda", dtype=torch.float64)
        k1, v1 = stored(s["k_new"]), stored(s["v_new"])
        for b in range(S):
            n = int(s["seq"][b])
            rows = s["table"][b, :-(-n // P)].long()
            kk = torch.cat([values("k", rows)[:, :n], k1[b, :, None]], 1)
            a = torch.softmax(s["q"][b].double().view(H, Q // H, D) @ kk.transpose(1, 2) / D ** 0.5, -1)
            del kk
            out[b] = (a @ torch.cat([values("v", rows)[:, :n], v1[b, :, None]], 1)).view(Q, D)
        if case["gate"]:
            out = out / (1 + torch.exp(-s["gate"].double()))[..., None]
        return (out, k1[:, None], v1[:, None]) if case["write"] else out
    k, v = s["k_out"].double(), s["v_out"].double()
    for b in range(S):
        n, at = int(s["count"][b]), int(s["start"][b])
        if n == 0:
            continue
        if case["op"] == "read":
            rows = s["table"][b, at // P:-(-(at + n) // P)].long()
            k[b, :n] = values("k", rows).transpose(0, 1)[at % P:at % P + n]
            v[b, :n] = values("v", rows).transpose(0, 1)[at % P:at % P + n]
            continue
        key, half = s["k_new"][b, :n], case["rotary"] // 2
        if half:
            turn = torch.polar(torch.ones(n, half, device="cuda", dtype=torch.float64),
                               torch.outer(torch.arange(at, at + n, device="cuda").double(),
                                           THETA ** (torch.arange(half, device="cuda").double() / -half)))
            z = torch.complex(key[..., :half].double(), key[..., half:2 * half].double()) * turn[:, None]
            key = torch.cat([z.real.to(torch.bfloat16), z.imag.to(torch.bfloat16), key[..., 2 * half:]], -1)
        k[b, :n], v[b, :n] = stored(key), stored(s["v_new"][b, :n])
    return k, v
