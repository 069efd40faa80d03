"""Measured cases of the long-context operators: decode over the pages that a
cheap score selects, the page summaries it scores, and linear attention with a
decay for each head (the chunked form for prompts, the recurrent form for
single tokens).

Each case is run in a plain form (elementary torch operations in 32 bits, the
page scores in 64) or, with `own` set, through the library's entry points.
Head layouts, page sizes and context lengths are those of the repository's
benchmark: 8 query / 2 KV heads of 256, 16 / 8 heads of 128, 24 / 4 heads of
256; 16- and 64-token pages; up to 1,048,576 cached tokens.
"""
import math
import random

import numpy as np
import torch

own = False

THETA = 5e6


def listed():
    return [
        # decode of one very long stream: the scores read one summary for each page
        {"name": "sparse 1 x 1048576", "op": "sparse", "streams": 1, "lo": 1048576, "hi": 1048576, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "rotary": 64, "page": 64, "pages": 64, "first": 1, "last": 2, "fp8": False,
         "gate": False, "write": False},
        # the long-context batch of the benchmark
        {"name": "sparse 8 x 262144", "op": "sparse", "streams": 8, "lo": 262144, "hi": 262144, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "rotary": 64, "page": 64, "pages": 64, "first": 1, "last": 2, "fp8": False,
         "gate": False, "write": False},
        # a full serving batch with ragged lengths in small pages; some streams have fewer pages than the budget
        {"name": "sparse 64 ragged", "op": "sparse", "streams": 64, "lo": 64, "hi": 4096, "q_heads": 16,
         "kv_heads": 8, "dim": 128, "rotary": 128, "page": 16, "pages": 32, "first": 1, "last": 4, "fp8": False,
         "gate": False, "write": False},
        # the same kind of batch over an E4M3 cache
        {"name": "sparse fp8 64 x 16384", "op": "sparse", "streams": 64, "lo": 15000, "hi": 16384, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "rotary": 64, "page": 16, "pages": 64, "first": 1, "last": 4, "fp8": True,
         "gate": True, "write": False},
        # one interactive stream, the new entry written back: latency counts
        {"name": "sparse 1 x 5003 write", "op": "sparse", "streams": 1, "lo": 5003, "hi": 5003, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "rotary": 64, "page": 16, "pages": 32, "first": 1, "last": 2, "fp8": False,
         "gate": True, "write": True},
        # summaries of the pages that a batch of prompts has just filled
        {"name": "summarize 64 x 4096", "op": "summarize", "streams": 64, "lo": 64, "hi": 4096, "q_heads": 16,
         "kv_heads": 8, "dim": 128, "page": 16, "fp8": False, "append": 4096},
        # the same after one decode step: at most one page a stream is completed
        {"name": "summarize step fp8", "op": "summarize", "streams": 64, "lo": 64, "hi": 4096, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "page": 16, "fp8": True, "append": 1},
        # recurrent steps: a serving batch, and one stream
        {"name": "linear step 64", "op": "step", "streams": 64, "q_heads": 16, "kv_heads": 8, "dim": 128,
         "gate": True, "write": True},
        {"name": "linear step 1", "op": "step", "streams": 1, "q_heads": 8, "kv_heads": 2, "dim": 256,
         "gate": True, "write": True},
        # prompts: one long one, a ragged batch, and the short ones of a chat turn
        {"name": "linear prompt 1 x 32768", "op": "prompt", "streams": 1, "lo": 32768, "hi": 32768, "q_heads": 16,
         "kv_heads": 8, "dim": 128, "gate": False},
        {"name": "linear prompt 16 ragged", "op": "prompt", "streams": 16, "lo": 512, "hi": 4096, "q_heads": 8,
         "kv_heads": 2, "dim": 256, "gate": True},
        {"name": "linear prompt 4 short", "op": "prompt", "streams": 4, "lo": 1, "hi": 150, "q_heads": 24,
         "kv_heads": 4, "dim": 256, "gate": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sparse", "sparse", "summarize", "step", "prompt", "prompt"])
    qh, kvh, dim = rng.choice([(8, 2, 256), (16, 8, 128), (24, 4, 256), (8, 8, 128), (6, 2, 128), (8, 1, 128), (5, 1, 256)])
    c = {"op": op, "q_heads": qh, "kv_heads": kvh, "dim": dim}
    streams = _log(rng, 1, 64)
    if op == "sparse":
        # at most 1,048,576 cached tokens of 2 x 256 over the batch, and one stream's table as long as the longest listed
        most = 1048576 * 512 // (kvh * dim)
        hi = _log(rng, 40, max(41, min(262144, most // streams)))
        page = rng.choice([16, 16, 32, 64, 24, 128])
        last = rng.randint(1, 4)
        c.update(streams=streams, lo=rng.choice([hi, max(1, hi // 8)]), hi=hi, rotary=rng.choice([dim, dim // 4, 0]),
                 page=page, pages=rng.randint(last + 2, 96), first=rng.randint(0, 2), last=last,
                 fp8=rng.random() < 0.3, gate=rng.random() < 0.5, write=hi * streams * kvh * dim < 1 << 23)
    elif op == "summarize":
        most = 262144 * 1024 // (kvh * dim)
        hi = _log(rng, 16, max(17, min(16384, most // streams)))
        c.update(streams=streams, lo=max(1, hi // 8), hi=hi, page=rng.choice([16, 32, 64, 24]), fp8=rng.random() < 0.3,
                 append=rng.choice([1, hi, max(1, hi // 3)]))
    elif op == "step":
        c.update(streams=streams, gate=rng.random() < 0.5, write=rng.random() < 0.8)
    else:
        most = 32768 * 2048 // (qh * dim)
        hi = _log(rng, 1, max(2, most // streams))
        c.update(streams=streams, lo=rng.choice([hi, max(1, hi // 8), 0]), hi=hi, gate=rng.random() < 0.5)
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


def _pool(g, pages, heads, page, dim, fp8):
    """A page pool: a page's entries share a direction, as neighbouring keys do."""
    out = torch.empty(pages, heads, page, dim, device="cuda", dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16)
    step = max(1, (1 << 27) // (heads * page * dim))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn(n, heads, page, dim, generator=g, device="cuda", dtype=torch.float32)
        x += torch.randn(n, heads, 1, dim, generator=g, device="cuda", dtype=torch.float32) * 0.5
        out[at:at + n] = x.to(out.dtype)
    return out


K_SCALE, V_SCALE = 0.75, 1.25  # of the E4M3 pools


def _log_decay(heads):
    """Decays 1 - 2^-(5 + h), as their logarithms: heads that forget over 32 tokens, over 64, ..."""
    return np.log1p(-np.exp2(-5.0 - np.arange(heads))).astype(np.float32)


def prepare(case, seed):
    g = _generator(seed)
    H, D, S = case["kv_heads"], case["dim"], case["streams"]
    s = {"case": case}
    if case["op"] in ("sparse", "summarize"):
        lens, P, fp8 = _lens(case), case["page"], case["fp8"]
        room = [n // P + 1 for n in lens]
        total = sum(room) + 3
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        at = torch.tensor([0] + room[:-1]).cumsum(0)[:, None] + torch.arange(max(room))[None]
        inside = torch.arange(max(room))[None] < torch.tensor(room)[:, None]
        table = torch.where(inside.cuda(), perm[at.clamp(max=total - 1).cuda()], -1).to(torch.int32).contiguous()
        k = _pool(g, total, H, P, D, fp8)
        s.update(k=k, table=table, seq=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        # a pool of values belongs to every cache; the summaries do not read it
        s["v"] = _pool(g, total, H, P, D, fp8) if case["op"] == "sparse" else torch.zeros_like(k)
        if case["op"] == "sparse":
            scale = K_SCALE if fp8 else 1.0
            s["summary"] = torch.empty(total, H, D, device="cuda", dtype=torch.bfloat16)
            for i in range(0, total, 4096):
                s["summary"][i:i + 4096] = (k[i:i + 4096].float().mean(2) * scale).to(torch.bfloat16)
            s.update(q=_normal(g, S, case["q_heads"], D), k_new=_normal(g, S, H, D), v_new=_normal(g, S, H, D),
                     gate=_normal(g, S, case["q_heads"]) if case["gate"] else None, pos=s["seq"].clone(),
                     out=torch.zeros(S, case["q_heads"], D, device="cuda"),
                     selected=torch.zeros(S, H, case["pages"], device="cuda", dtype=torch.int32))
        else:
            n = torch.tensor(lens, dtype=torch.int32)
            start = (n - case["append"]).clamp(min=0)
            s.update(start=start.cuda(), count=(n - start).cuda(),
                     summary=torch.zeros(total, H, D, device="cuda", dtype=torch.bfloat16))
    else:
        s["log_decay"] = torch.from_numpy(_log_decay(H)).cuda()
        # a state that has run for a while: its entries have the size of a sum over the decay's reach
        reach = (1 / (1 - (2 * s["log_decay"].double()).exp())).sqrt().float()
        s["state"] = torch.randn(S, H, D, D, generator=g, device="cuda") * reach[None, :, None, None]
        if case["op"] == "step":
            s.update(q=_normal(g, S, case["q_heads"], D), k=_normal(g, S, H, D), v=_normal(g, S, H, D),
                     gate=_normal(g, S, case["q_heads"]) if case["gate"] else None,
                     pos=torch.full((S,), 1000, dtype=torch.int32, device="cuda"),
                     out=torch.zeros(S, case["q_heads"], D, device="cuda"))
        else:
            T = case["hi"]
            s.update(q=_normal(g, S, T, case["q_heads"], D), k=_normal(g, S, T, H, D), v=_normal(g, S, T, H, D),
                     gate=_normal(g, S, T, case["q_heads"]) if case["gate"] else None,
                     count=torch.tensor(_lens(case), dtype=torch.int32, device="cuda"),
                     start=torch.zeros(S, dtype=torch.int32, device="cuda"),
                     out=torch.zeros(S, T, case["q_heads"], D, device="cuda"))
    if own:
        import decode_attention_kv_dattn_gb300 as dattn
        if case["op"] in ("sparse", "summarize"):
            layer = {"kind": dattn.CACHE_PAGED, "page_size": P, "rotary_dim": case.get("rotary", 0), "rope_theta": THETA}
            if fp8:
                layer.update(kv_format=dattn.KV_E4M3, k_scale=K_SCALE, v_scale=V_SCALE)
            s["handle"] = dattn.Handle(case["q_heads"], H, D, [layer], S, max_context=max(lens),
                                       max_selected_pages=case.get("pages", 0))
            s["cache"] = dattn.paged_cache(s["k"], s["v"], s["table"], s["seq"])
        else:
            s["handle"] = dattn.Handle(case["q_heads"], H, D, [{"kind": dattn.CACHE_STATE, "log_decay": _log_decay(H)}], S)
            s["cache"] = dattn.state_cache(s["state"])
    return s


# ---------------------------------------------------------------- plain forms

def _rotated(x, pos, rotary):
    """x [B, heads, D] in 64 bits, the first `rotary` dims turned at pos [B] in pairs (i, i + rotary / 2)."""
    x = x.double()
    if not rotary:
        return x
    half = rotary // 2
    freq = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) * 2 / rotary)
    angle = (pos.double()[:, None] * freq)[:, None]
    c, s = angle.cos(), angle.sin()
    a, b = x[..., :half], x[..., half:rotary]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., rotary:]], -1)


def _keys(s, pages):
    """The K and V of the given pages (of their own KV head each) in 32 bits, scales applied."""
    case = s["case"]
    heads = torch.arange(case["kv_heads"], device="cuda")[None, :, None]
    k, v = s["k"][pages, heads].float(), s["v"][pages, heads].float()
    return (k * K_SCALE, v * V_SCALE) if case["fp8"] else (k, v)


def _sparse(s):
    case = s["case"]
    B, H, D, P = case["streams"], case["kv_heads"], case["dim"], case["page"]
    G, budget = case["q_heads"] // H, case["pages"]
    n = s["seq"].long()
    pages = (n + P - 1) // P
    table = s["table"].long()
    at = torch.arange(table.shape[1], device="cuda")
    # 64 bits: two pages' scores may lie as near as one likes, and the selection is a border between them
    q = _rotated(s["q"], s["pos"], case["rotary"]).view(B, H, G, D)
    means = s["summary"][table.clamp(min=0)].double()
    score = torch.einsum("bhgd,bphd->bhgp", q, means).amax(2)
    keep = (at < case["first"]) | (at >= pages[:, None] - case["last"])
    score = torch.where(keep[:, None], math.inf, score)
    score = torch.where(at < pages[:, None, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    chosen = torch.where(order < pages[:, None, None], order, table.shape[1]).sort(-1).values
    if chosen.shape[-1] < budget:
        chosen = torch.nn.functional.pad(chosen, (0, budget - chosen.shape[-1]), value=table.shape[1])
    real = chosen < table.shape[1]
    selected = torch.where(real, chosen, -1).to(torch.int32)
    physical = torch.gather(table[:, None].expand(-1, H, -1), 2, chosen.clamp(max=table.shape[1] - 1)).clamp(min=0)
    k, v = _keys(s, physical)
    valid = (chosen[..., None] * P + torch.arange(P, device="cuda") < n[:, None, None, None]) & real[..., None]
    k_new = _rotated(s["k_new"], s["pos"], case["rotary"]).to(torch.bfloat16)
    v_new = s["v_new"]
    if case["fp8"]:
        k_new = (k_new.double() / K_SCALE).clamp(-448, 448).float().to(torch.float8_e4m3fn)
        v_new = (v_new.double() / V_SCALE).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    kn, vn = (k_new.float() * K_SCALE, v_new.float() * V_SCALE) if case["fp8"] else (k_new.float(), v_new.float())
    v = torch.where(valid[..., None], v, 0).view(B, H, -1, D)
    q32 = (q / math.sqrt(D)).float()
    a = torch.einsum("bhgd,bhnd->bhgn", q32, k.view(B, H, -1, D))
    a = torch.where(valid.view(B, H, 1, -1), a, -math.inf)
    a = torch.cat([a, torch.einsum("bhgd,bhd->bhg", q32, kn)[..., None]], -1)
    a = (a - a.amax(-1, keepdim=True)).exp()
    a = a / a.sum(-1, keepdim=True)
    out = torch.einsum("bhgn,bhnd->bhgd", a, torch.cat([v, vn[:, :, None]], 2)).reshape(B, H * G, D)
    if case["gate"]:
        out = out / (1 + (-s["gate"].float()).exp())[..., None]
    if case["write"]:
        rows, off = table[torch.arange(B, device="cuda"), n // P], n % P
        s["k"][rows, :, off] = k_new
        s["v"][rows, :, off] = v_new
    return out, selected


def _summarize(s):
    case = s["case"]
    P = case["page"]
    at = torch.arange(s["table"].shape[1], device="cuda")
    # the pages whose last token is among the new ones
    done = (at >= (s["start"] // P)[:, None]) & (at < ((s["start"] + s["count"]) // P)[:, None])
    rows = s["table"].long()[done]
    mean = s["k"][rows].float().sum(2) / P
    s["summary"][rows] = (mean * K_SCALE if case["fp8"] else mean).to(torch.bfloat16)
    return s["summary"]


def _step(s):
    case = s["case"]
    B, H, D = case["streams"], case["kv_heads"], case["dim"]
    state = s["state"] * s["log_decay"].double().exp().float()[None, :, None, None]
    state = state + s["k"].float()[..., None] * s["v"].float()[:, :, None]
    out = torch.einsum("bhgd,bhde->bhge", s["q"].float().view(B, H, -1, D), state) / math.sqrt(D)
    out = out.reshape(B, -1, D)
    if case["gate"]:
        out = out / (1 + (-s["gate"].float()).exp())[..., None]
    if case["write"]:
        s["state"].copy_(state)
    return out, s["state"]


def _prompt(s, chunk=128):
    case = s["case"]
    S, T, H, D = case["streams"], case["hi"], case["kv_heads"], case["dim"]
    G, N = case["q_heads"] // H, -(-T // chunk)
    g = s["log_decay"].double()
    live = torch.arange(T, device="cuda") < s["count"][:, None]
    pad = (0, 0, 0, 0, 0, N * chunk - T)
    cut = lambda x: torch.nn.functional.pad(x, pad).view(S, N, chunk, H, -1, D)  # noqa: E731
    k32 = torch.where(live[..., None, None], s["k"].float(), 0)
    v32 = s["v"].float()
    q, k, v = cut(s["q"].float()), cut(k32)[:, :, :, :, 0], cut(v32)[:, :, :, :, 0]
    i = torch.arange(chunk, device="cuda", dtype=torch.float64)
    lag = i[:, None] - i
    near = torch.where(lag >= 0, (g[:, None, None] * lag.clamp(min=0)).exp(), 0).float()
    a = torch.einsum("snihgd,snjhd->snhgij", q, k) * near[:, None]
    out = torch.einsum("snhgij,snjhd->snihgd", a, v)
    # the state at the start of each chunk: the first one's, decayed, and the sums of the chunks between
    sums = torch.einsum("snjhd,hj,snjhe->snhde", k, (g[:, None] * (chunk - 1 - i)).exp().float(), v)
    m = torch.arange(N, device="cuda", dtype=torch.float64) * chunk
    gap = m[:, None] - m - chunk
    far = torch.where(gap >= 0, (g[:, None, None] * gap.clamp(min=0)).exp(), 0).float()
    states = torch.einsum("hnm,smhde->snhde", far, sums)
    states = states + torch.einsum("hn,shde->snhde", (g[:, None] * m).exp().float(), s["state"])
    out = out + torch.einsum("snihgd,snhde->snihge", q, states) * (g * (i[:, None] + 1)).exp().float()[None, None, :, :, None, None]
    out = out.reshape(S, N * chunk, H * G, D)[:, :T] / math.sqrt(D)
    if case["gate"]:
        out = out / (1 + (-s["gate"].float()).exp())[..., None]
    # the state after each stream's last token
    n = s["count"].double()
    back = (n[:, None] - 1 - torch.arange(T, device="cuda", dtype=torch.float64)).clamp(min=0)
    w = (back[..., None] * g).exp().float()
    state = torch.einsum("sthd,sthe->shde", k32 * w[..., None], v32)
    s["state"].copy_(state + s["state"] * (n[:, None] * g).exp().float()[..., None, None])
    return torch.where(live[..., None, None], out, s["out"]), s["state"]


def _pools(s):
    """The pools as the values they stand for (a scaled E4M3 value has few enough bits for bf16)."""
    if not s["case"]["fp8"]:
        return s["k"], s["v"]
    return s["k"].to(torch.bfloat16) * K_SCALE, s["v"].to(torch.bfloat16) * V_SCALE


def run(s):
    case = s["case"]
    if case["op"] == "sparse":
        if own:
            s["handle"].sparse_decode(0, s["cache"], s["summary"], s["q"], s["k_new"], s["v_new"], s["pos"], s["out"],
                                      case["pages"], keep_first=case["first"], keep_last=case["last"], gate=s["gate"],
                                      write_back=case["write"], selected=s["selected"])
            out, selected = s["out"], s["selected"]
        else:
            out, selected = _sparse(s)
        # the pools are outputs where the new entry is written to them
        return (out, selected, *_pools(s)) if case["write"] else (out, selected)
    if case["op"] == "summarize":
        if own:
            s["handle"].summarize(0, s["cache"], s["summary"], s["start"], s["count"], max_tokens=case["append"])
            return s["summary"]
        return _summarize(s)
    if case["op"] == "step":
        if own:
            s["handle"].decode(0, s["cache"], s["q"], s["k"], s["v"], s["pos"], s["out"], gate=s["gate"],
                               write_back=case["write"])
            return s["out"], s["state"]
        return _step(s)
    if own:
        s["handle"].prefill(0, s["cache"], s["q"], s["k"], s["v"], s["count"], s["start"], s["out"], gate=s["gate"])
        return s["out"], s["state"]
    return _prompt(s)


def work(case):
    H, D, S, Q = case["kv_heads"], case["dim"], case["streams"], case["q_heads"]
    if case["op"] in ("sparse", "summarize"):
        P, size, lens = case["page"], 1 if case["fp8"] else 2, _lens(case)
    if case["op"] == "sparse":
        pages = [-(-n // P) for n in lens]
        # a stream with no more pages than the budget needs no score
        scored = [p - case["first"] - case["last"] if p > case["pages"] else 0 for p in pages]
        read = [n if p <= case["pages"] else (case["pages"] - 1) * P + (n - 1) % P + 1 for n, p in zip(lens, pages)]
        io = S * ((Q + 2 * H) * D * 2 + Q * D * 4 + H * case["pages"] * 4) + sum(pages) * 4
        if case["write"]:
            io += S * 2 * H * D * size
        return {"bytes": io + sum(scored) * H * D * 2 + sum(read) * H * D * 2 * size,
                "flops": sum(scored) * Q * D * 2 + sum(read) * Q * D * 4}
    if case["op"] == "summarize":
        done = sum(n // P - max(0, n - case["append"]) // P for n in lens)
        return {"bytes": done * H * D * (P * size + 2) + S * 8 + done * 4, "flops": done * H * D * P}
    if case["op"] == "step":
        io = S * ((Q + 2 * H) * D * 2 + Q * D * 4)
        return {"bytes": io + S * H * D * D * 4 * (2 if case["write"] else 1), "flops": S * H * D * D * 3 + S * Q * D * D * 2}
    # the products with the state (the recurrence's own count): what the chunked form adds inside a chunk is its choice
    T = sum(_lens(case))
    return {"bytes": T * ((Q + 2 * H) * D * 2 + Q * D * 4) + S * H * D * D * 8, "flops": T * (H + Q) * D * D * 2}


# ---------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    H, D, S, Q = case["kv_heads"], case["dim"], case["streams"], case["q_heads"]
    group = Q // H
    sigmoid = lambda x: 1 / (1 + torch.exp(-x.double()))  # noqa: E731
    if case["op"] == "step":
        old = s["state"].double() * torch.exp(s["log_decay"].double()).view(1, H, 1, 1)
        new = old + s["k"].double().unsqueeze(3) * s["v"].double().unsqueeze(2)
        out = (s["q"].double().unsqueeze(3) * new.repeat_interleave(group, 1)).sum(2) / D ** 0.5
        if case["gate"]:
            out = out * sigmoid(s["gate"]).unsqueeze(2)
        return out, new if case["write"] else s["state"].double()
    if case["op"] == "prompt":
        # token by token, as the recurrence defines it
        state, out = s["state"].double(), s["out"].double()
        decay = torch.exp(s["log_decay"].double()).view(1, H, 1, 1)
        for t in range(case["hi"]):
            on = (t < s["count"]).view(S, 1, 1, 1)
            new = state * decay + s["k"][:, t].double().unsqueeze(3) * s["v"][:, t].double().unsqueeze(2)
            state = torch.where(on, new, state)
            o = torch.matmul(s["q"][:, t].double().view(S, H, group, D), state).view(S, Q, D) / D ** 0.5
            if case["gate"]:
                o = o * sigmoid(s["gate"][:, t]).unsqueeze(2)
            out[:, t] = torch.where(on[:, 0], o, out[:, t])
        return out, state
    P = case["page"]
    k_scale, v_scale = (K_SCALE, V_SCALE) if case["fp8"] else (1.0, 1.0)
    if case["op"] == "summarize":
        want = s["summary"].double()
        for b in range(S):
            lo, hi = int(s["start"][b]), int(s["start"][b] + s["count"][b])
            if hi // P > lo // P:
                rows = s["table"][b, lo // P:hi // P].long()
                want[rows] = s["k"][rows].double().mean(2) * k_scale
        return want

    def turn(x, pos):
        x, half = x.double().clone(), case["rotary"] // 2
        if half:
            z = torch.complex(x[:, :half], x[:, half:2 * half])
            w = torch.arange(half, device=x.device).double().mul(-2.0 / case["rotary"])
            z = z * torch.polar(torch.ones_like(w), pos * THETA ** w)
            x[:, :half], x[:, half:2 * half] = z.real, z.imag
        return x

    out = torch.empty(S, Q, D, device="cuda", dtype=torch.float64)
    selected = torch.full((S, H, case["pages"]), -1, device="cuda", dtype=torch.int32)
    for b in range(S):
        n = int(s["seq"][b])
        m = -(-n // P)
        rows = s["table"][b, :m].long()
        qr, kr = turn(s["q"][b], int(s["pos"][b])), turn(s["k_new"][b], int(s["pos"][b])).to(torch.bfloat16)
        for h in range(H):
            qh = qr[h * group:(h + 1) * group]
            pick = list(range(m))
            if m > case["pages"]:
                forced = set(range(case["first"])) | set(range(m - case["last"], m))
                best = (s["summary"][rows, h].double() @ qh.T).max(1).values.tolist()
                rest = sorted((p for p in range(m) if p not in forced), key=lambda p: (-best[p], p))
                pick = sorted(forced | set(rest[:case["pages"] - len(forced)]))
            selected[b, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            at = rows[torch.tensor(pick, dtype=torch.long, device="cuda")]
            left = n - (len(pick) - 1) * P if not pick else n - pick[-1] * P
            size = max(0, (len(pick) - 1) * P + left) if pick else 0
            kk = s["k"][at, h].double().reshape(-1, D)[:size] * k_scale
            vv = s["v"][at, h].double().reshape(-1, D)[:size] * v_scale
            k1, v1 = kr[h].double(), s["v_new"][b, h].double()
            if case["fp8"]:
                k1 = (k1 / k_scale).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() * k_scale
                v1 = (v1 / v_scale).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() * v_scale
            kk, vv = torch.cat([kk, k1[None]]), torch.cat([vv, v1[None]])
            o = torch.softmax(qh @ kk.T / D ** 0.5, 1) @ vv
            out[b, h * group:(h + 1) * group] = o
            if case["write"]:
                page, off = int(s["table"][b, n // P]), n % P
                s["k"][page, h, off] = (k1 / k_scale).to(s["k"].dtype)
                s["v"][page, h, off] = (v1 / v_scale).to(s["v"].dtype)
    if case["gate"]:
        out = out * sigmoid(s["gate"]).unsqueeze(2)
    return (out, selected, s["k"].double() * k_scale, s["v"].double() * v_scale) if case["write"] else (out, selected)
