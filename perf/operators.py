"""Timed cases of the paged KV cache operators, with a plain PyTorch form of each.

Three operators share one cache layout: `paged_append` (rotates and writes new keys and values), `paged_attend`
(exact softmax attention over the cache, whole or restricted to a support) and `paged_gather` (reads rows back as
dense bf16).  A cache is a pool of pages; `page_table[b, i]` names the page that holds tokens [i * page, (i + 1) * page)
of sequence b, and `kv_len[b]` counts its tokens, the newest included.

bf16 cache: [pages, Hkv, page, 2, d], a token's key then its value.
4-bit cache: uint8 [pages, Hkv, page, d + 16], per token d/2 bytes of key codes, d/2 of value codes, 4 bf16 key scales,
4 bf16 value scales.  A row of d values has 4 groups of d/4 consecutive channels; a value is scale * (code - 8).
Where channel c = g * d/4 + j sits:
  keys    byte (t * d/8 + g * d/32 + e // 2), nibble e % 2 (0 low), with t = j // (d/16), e = j % (d/16)
  values  byte ((j % 8) * d/16 + g * d/64 + j // 16), low nibble for j % 16 < 8, else high
Rounding: scale = amax / 7 rounded up to bf16, code - 8 = x / scale rounded to nearest even (fp32), in [-7, 7].
"""
import math

import torch

own = False

BF16, INT4 = "bf16", "int4"


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 32 sequences of a serving batch: latency of the decode step's first operator
        _append("append_step", B=32, n=1, n_max=131072, Hq=32, Hkv=8, d=128, page=16, fmt=INT4, rot=128),
        # a 4096-token prefill chunk behind 28672 cached tokens, written as 4 bits
        _append("append_chunk", B=1, n=4096, n_max=32768, Hq=32, Hkv=8, d=128, page=64, fmt=INT4, rot=128),
        # prompts of several lengths in one call, bf16 pages, interleaved rotation of half the channels, odd counts
        _append("append_prompts_bf16", B=7, n=1999, n_max=9001, Hq=16, Hkv=2, d=64, page=32, fmt=BF16, rot=32,
                ragged=True, interleaved=True),
        # the cached prefix of a chunked prefill, read back for the dense prefill kernels
        _gather("gather_prefix", B=1, n_max=28672, Hkv=8, d=128, page=64, fmt=INT4),
        # a ragged batch of short bf16 sequences
        _gather("gather_batch_bf16", B=8, n_max=9001, Hkv=2, d=64, page=16, fmt=BF16, ragged=True),
        # one short sequence of a small model: latency
        _attend("attend_short", B=1, n_max=4096, Hq=4, Hkv=1, d=64, page=16, fmt=INT4),
        # a serving batch of many sequences of different lengths, one of them empty
        _attend("attend_batch", B=64, n_max=9001, Hq=32, Hkv=8, d=128, page=16, fmt=INT4, ragged=True),
        # long contexts
        _attend("attend_128k", B=4, n_max=131072, Hq=32, Hkv=4, d=128, page=64, fmt=INT4),
        # the same from bf16 pages
        _attend("attend_64k_bf16", B=4, n_max=65536, Hq=32, Hkv=4, d=128, page=64, fmt=BF16),
        # five drafted tokens of each sequence checked at once
        _attend("attend_draft", B=16, n=5, n_max=9001, Hq=32, Hkv=8, d=128, page=32, fmt=INT4, ragged=True),
        # a prefill chunk against a 4-bit prefix
        _attend("attend_chunk", B=1, n=1024, n_max=28672, Hq=32, Hkv=8, d=128, page=64, fmt=INT4),
        # sparse decode: a support of 12288 single tokens for each kv head of a 128K cache
        _attend("attend_support", B=4, n_max=131072, Hq=32, Hkv=4, d=128, page=64, fmt=INT4, cap=12288),
    ]


def _append(name, B, n, n_max, Hq, Hkv, d, page, fmt, rot, ragged=False, interleaved=False):
    c = dict(op="append", B=B, n=n, n_max=n_max, Hq=Hq, Hkv=Hkv, d=d, page=page, fmt=fmt, rot=rot, ragged=ragged,
             interleaved=interleaved)
    return dict(c, name=name) if name else c


def _gather(name, B, n_max, Hkv, d, page, fmt, ragged=False):
    c = dict(op="gather", B=B, n_max=n_max, Hkv=Hkv, d=d, page=page, fmt=fmt, ragged=ragged)
    return dict(c, name=name) if name else c


def _attend(name, B, n_max, Hq, Hkv, d, page, fmt, n=1, ragged=False, cap=0, unit=1):
    c = dict(op="attend", B=B, n=n, n_max=n_max, Hq=Hq, Hkv=Hkv, d=d, page=page, fmt=fmt, ragged=ragged, cap=cap,
             unit=unit)
    return dict(c, name=name) if name else c


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["append", "append", "gather", "attend", "attend", "attend", "support"])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    fmt = rng.choice([INT4, INT4, BF16])
    B = between(1, 64)
    ragged = rng.random() < 0.5
    if kind == "append":
        G = rng.choice([1, 2, 4, 8])
        n = between(1, 4096)
        B = max(1, min(B, 4096 // n))
        room = (1 << 29) // (B * Hkv * 4 * d)              # tokens of a sequence in a pool of half a GiB
        n_max = min(n + between(1, 120000), max(n, room))
        return _append(None, B, n, n_max, G * Hkv, Hkv, d, page, fmt, rng.choice([16, 32, d // 2, d]), ragged,
                       rng.random() < 0.3)
    rows = 1 << 21 if fmt == INT4 else 1 << 20            # cached rows (tokens x kv heads) of the largest case
    if kind == "gather":
        rows //= 8
    n_max = between(1, min(131072, rows // Hkv))
    B = max(1, min(B, rows // (n_max * Hkv)))
    if kind == "gather":
        return _gather(None, B, n_max, Hkv, d, page, fmt, ragged)
    G = rng.choice([1, 2, 3, 4, 6, 8, 16])
    if kind == "support":
        unit = rng.choice([1, 1, 16, 64])
        return _attend(None, B, n_max, G * Hkv, Hkv, d, page, fmt, 1, ragged, max(1, n_max // unit // between(2, 20)),
                       unit)
    n = rng.choice([1, 1, 1, 2, 4, 7, between(8, 512)])
    n = max(1, min(n, n_max, int(4.5e11 / (4.0 * d * G * Hkv * B * n_max))))
    return _attend(None, B, n_max, G * Hkv, Hkv, d, page, fmt, n, ragged)


def _lens(c):
    """Tokens of each sequence after the call, and how many of them are new (one of a large ragged batch is empty)."""
    B, n = c["B"], c.get("n", 0)
    if not c["ragged"]:
        return [c["n_max"]] * B, [n] * B
    lens, new = [], []
    for b in range(B):
        f = (b + 1) * 0.6180339887498949 % 1.0
        k = n if c["op"] == "attend" or b == 0 else max(1, int(n * f))
        L = c["n_max"] if b == 0 else max(k, int(c["n_max"] * f))
        if B >= 4 and b == B // 2:
            L = k = 0
        lens.append(L)
        new.append(k)
    return lens, new


def work(case):
    c = case
    lens, new = _lens(c)
    d, Hkv = c["d"], c["Hkv"]
    row = d + 16 if c["fmt"] == INT4 else 4 * d            # bytes of a token's key and value, per kv head
    if c["op"] == "append":
        T, Hq = sum(new), c["Hq"]
        b = T * (2 * Hq * d * 2 + 2 * Hkv * d * 2 + Hkv * row)
        if c["fmt"] == INT4:                               # read back: the rows, as dense bf16
            b += T * Hkv * (row + 4 * d)
        return {"bytes": b, "flops": T * (Hq + Hkv) * c["rot"] * 3}
    if c["op"] == "gather":
        T = sum(lens)
        return {"bytes": T * Hkv * (row + 4 * d), "flops": T * Hkv * d * 2}
    Hq, G = c["Hq"], c["Hq"] // Hkv
    T = sum(new)
    if c["cap"]:
        rows = sum(min(L, min(c["cap"], -(-L // c["unit"])) * c["unit"]) for L in lens)
        return {"bytes": rows * Hkv * row + c["B"] * Hkv * c["cap"] * 4 + T * Hq * (4 * d + 4),
                "flops": rows * Hkv * G * d * 4}
    pairs = sum(k * L - k * (k - 1) // 2 for L, k in zip(lens, new))
    return {"bytes": sum(lens) * Hkv * row + T * Hq * (4 * d + 4), "flops": pairs * Hq * d * 4}


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    lens, new = _lens(c)
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    width = max(1, -(-max(lens) // page))
    P = B * width + 3                                       # a few pages belong to nobody
    perm = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    s = {"case": c, "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "page_table": perm[: B * width].reshape(B, width).contiguous()}
    start = [0]
    for k in new:
        start.append(start[-1] + k)
    T = start[-1]
    uniform_one = all(k == 1 for k in new)
    s["seq_start"] = None if uniform_one else torch.tensor(start, dtype=torch.int32, device="cuda")
    if c["op"] == "append":
        # the model's fused projection output: q, k and v of a token are slices of one row
        qkv = randn(T, c["Hq"] + 2 * Hkv, d).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, : c["Hq"]], qkv[:, c["Hq"]: c["Hq"] + Hkv], qkv[:, c["Hq"] + Hkv:]
        half = c["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        s["N"] = max(new)
        s["first"] = (s["kv_len"] - torch.tensor(new, dtype=torch.int32, device="cuda")).contiguous()
        s["cache"] = _empty(P, c)
        s["K"] = torch.zeros(B, Hkv, s["N"], d, dtype=torch.bfloat16, device="cuda")
        s["V"] = torch.zeros_like(s["K"])
    else:
        s["cache"] = _empty(P, c)
        for i in range(0, P, max(1, (1 << 17) // (page * Hkv))):   # a block of pages at a time keeps the scratch small
            part = s["cache"][i: i + max(1, (1 << 17) // (page * Hkv))]
            kv = randn(2, part.shape[0], Hkv, page, d)
            kv *= torch.exp(0.5 * randn(2, part.shape[0], Hkv, page, 1))   # token norms vary
            part.copy_(_pack(kv[0], kv[1]) if c["fmt"] == INT4 else kv.permute(1, 2, 3, 0, 4))
    if c["op"] == "gather":
        s["K"] = torch.zeros(B, Hkv, c["n_max"], d, dtype=torch.bfloat16, device="cuda")
        s["V"] = torch.zeros_like(s["K"])
    if c["op"] == "attend":
        s["q"] = randn(T, c["Hq"], d).to(torch.bfloat16)
        s["sm_scale"] = d ** -0.5
        s["idx"] = s["count"] = None
        if c["cap"]:
            # ascending supports, as the selection writes them: every unit's last and first blocks and random others
            U, M = B * Hkv, max(1, -(-max(lens) // c["unit"]))
            idx = torch.zeros(U, c["cap"], dtype=torch.int32, device="cuda")
            count = torch.zeros(U, dtype=torch.int32, device="cuda")
            for u in range(U):
                M = -(-lens[u // Hkv] // c["unit"])
                k = min(c["cap"], M)
                pick = torch.randperm(M, generator=gen, device="cuda")[:k]
                idx[u, :k] = pick.sort().values.to(torch.int32)
                count[u] = k
            s["idx"], s["count"] = idx, count
    if own:
        s["plan"] = _plans(s)
    return s


def _plans(s):
    """What a serving loop keeps: the calls' arguments, outputs and workspaces, built once."""
    import long_context_sparse_spa_b200 as spa

    c = s["case"]
    paged = dict(cache=s["cache"], page_table=s["page_table"], kv_len=s["kv_len"])
    if c["op"] == "append":
        add = spa.paged_append(k=s["k"], v=s["v"], q=s["q"], seq_start=s["seq_start"], inv_freq=s["inv_freq"],
                               interleaved=c["interleaved"], run=False, **paged)
        if c["fmt"] == BF16:
            return (add,)
        return add, spa.paged_gather(N=s["N"], start=s["first"], K=s["K"], V=s["V"], run=False, **paged)
    if c["op"] == "gather":
        return (spa.paged_gather(N=c["n_max"], K=s["K"], V=s["V"], run=False, **paged),)
    return (spa.paged_attend(q=s["q"], seq_start=s["seq_start"], sm_scale=s["sm_scale"], idx=s["idx"],
                             count=s["count"], unit_tokens=c["unit"], run=False, **paged),)


def _empty(P, c):
    if c["fmt"] == INT4:
        return torch.zeros(P, c["Hkv"], c["page"], c["d"] + 16, dtype=torch.uint8, device="cuda")
    return torch.zeros(P, c["Hkv"], c["page"], 2, c["d"], dtype=torch.bfloat16, device="cuda")


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        for p in s["plan"]:
            p.run()
        p = s["plan"][0]
        if c["op"] == "append":
            return (p.q_out, s["cache"]) if c["fmt"] == BF16 else (p.q_out, s["K"], s["V"])
        return (s["K"], s["V"]) if c["op"] == "gather" else (p.out, p.lse)
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "gather":
        K, V = _rows(s, c["n_max"])
        live = (torch.arange(c["n_max"], device="cuda") < s["kv_len"][:, None])[:, None, :, None]
        s["K"].copy_(torch.where(live, K, s["K"].float()))
        s["V"].copy_(torch.where(live, V, s["V"].float()))
        return s["K"], s["V"]
    return _plain_attend(s)


def _places(s):
    """Sequence and position of every new token."""
    T = s["k"].shape[0] if "k" in s else s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    if s["seq_start"] is None:
        return t, s["kv_len"].long() - 1
    start = s["seq_start"].long()
    b = torch.searchsorted(start, t, right=True) - 1
    return b, s["kv_len"].long()[b] - start[b + 1] + t


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _quantise(x):
    """Codes minus 8 and scales of rows [..., d] fp32."""
    d = x.shape[-1]
    g = x.reshape(*x.shape[:-1], 4, d // 4)
    top = g.abs().amax(-1)
    up = (top / torch.full_like(top, 7.0)).view(torch.int32)   # by a number, torch would multiply by a rounded 1/7
    scale = ((up + 0xFFFF) & ~0xFFFF).view(torch.float32)   # towards larger bf16
    code = torch.where(scale[..., None] > 0, torch.round(g / scale[..., None]), torch.zeros_like(g))
    return code.reshape(x.shape), scale


def _plain_append(s):
    c = s["case"]
    b, pos = _places(s)
    ang = pos.double()[:, None] * s["inv_freq"].double()    # 32 bits would lose the angles of far positions
    cos, sin = ang.cos().float(), ang.sin().float()
    q = _rotate(s["q"].float(), cos, sin, c["interleaved"]).to(torch.bfloat16)
    k, v = _rotate(s["k"].float(), cos, sin, c["interleaved"]), s["v"].float()
    if c["fmt"] == BF16:
        page = s["page_table"].long()[b, pos // c["page"]]
        s["cache"][page, :, pos % c["page"]] = torch.stack((k, v), 2).to(torch.bfloat16)
        return q, s["cache"]
    for out, x in ((s["K"], k), (s["V"], v)):
        code, scale = _quantise(x)
        out[b, :, pos - s["first"].long()[b]] = (code * scale.repeat_interleave(c["d"] // 4, -1)).to(torch.bfloat16)
    return q, s["K"], s["V"]


def _code_places(d):
    """Flat nibble position (2 * byte + high) of every key and value channel within a row's codes."""
    ch = torch.arange(d, device="cuda")
    g, j = ch // (d // 4), ch % (d // 4)
    t, e = j // (d // 16), j % (d // 16)
    kpos = 2 * (t * (d // 8) + g * (d // 32) + e // 2) + e % 2
    vpos = 2 * ((j % 8) * (d // 16) + g * (d // 64) + j // 16) + (j % 16) // 8
    return kpos, vpos


def _pack(k, v):
    """Rows [..., d] fp32 as 4-bit cache rows [..., d + 16]."""
    d = k.shape[-1]
    parts, scales = [], []
    for x, place in zip((k, v), _code_places(d)):
        code, scale = _quantise(x)
        nib = torch.empty_like(code, dtype=torch.uint8)
        nib[..., place] = (code + 8).to(torch.uint8)
        parts.append(nib[..., 0::2] | (nib[..., 1::2] << 4))
        scales.append(scale.to(torch.bfloat16).contiguous().view(torch.uint8))
    return torch.cat(parts + scales, -1)


def _unpack(rows, dtype):
    """Keys and values [..., d] that 4-bit cache rows [..., d + 16] stand for."""
    d = rows.shape[-1] - 16
    out = []
    for i, place in enumerate(_code_places(d)):
        by = rows[..., i * d // 2: (i + 1) * d // 2]
        nib = torch.stack((by & 15, by >> 4), -1).flatten(-2)[..., place]
        scale = rows[..., d + 8 * i: d + 8 * i + 8].contiguous().view(torch.bfloat16)
        out.append((nib.to(dtype) - 8) * scale.to(dtype).repeat_interleave(d // 4, -1))
    return out


def _rows(s, n, dtype=torch.float32):
    """Keys and values [B, Hkv, n, d] of the first n tokens of every sequence (past its length: anything)."""
    c = s["case"]
    pages = -(-n // c["page"])
    x = s["cache"][s["page_table"][:, :pages].long()].transpose(1, 2)       # [B, Hkv, pages, page, ...]
    x = x.flatten(2, 3)[:, :, :n]
    if c["fmt"] == INT4:
        return _unpack(x, dtype)
    return x[..., 0, :].to(dtype), x[..., 1, :].to(dtype)


def _plain_attend(s):
    c = s["case"]
    B, Hkv, d, n = c["B"], c["Hkv"], c["d"], c["n_max"]
    G = c["Hq"] // Hkv
    K, V = _rows(s, n)
    b, pos = _places(s)
    new = c["n"]
    # queries as [B, Hkv, new, G, d]; a sequence without queries keeps zeros and is dropped again below
    i = pos - s["kv_len"].long()[b] + new
    have = i >= 0                                           # without seq_start an empty sequence still has a query row
    i = i.clamp(min=0)
    q = torch.zeros(B, new, Hkv, G, d, device="cuda")
    q[b, i] = s["q"].float().reshape(-1, Hkv, G, d)
    q = q.permute(0, 2, 1, 3, 4)
    n_idx = torch.arange(n, device="cuda")
    limit = s["kv_len"].long()[:, None] - new + 1 + torch.arange(new, device="cuda")      # keys each query may see
    mask = n_idx < limit[:, :, None]                        # [B, new, n]
    mask = mask[:, None, :, None, :]
    if c["cap"]:
        M = -(-n // c["unit"])
        on = torch.zeros(B * Hkv, M + 1, dtype=torch.bool, device="cuda")
        live = torch.arange(c["cap"], device="cuda") < s["count"][:, None]
        on.scatter_(1, torch.where(live, s["idx"].long(), torch.full_like(s["idx"].long(), M)), True)
        on = on[:, :M].repeat_interleave(c["unit"], 1)[:, :n].reshape(B, Hkv, 1, 1, n)
        mask = mask & on
    x = torch.matmul(q.flatten(2, 3), K.transpose(2, 3)).reshape(B, Hkv, new, G, n) * s["sm_scale"]
    x = x.masked_fill_(~mask, float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x = (x - m).exp_()
    z = x.sum(-1, keepdim=True)
    out = torch.matmul(x.flatten(2, 3), V).reshape(B, Hkv, new, G, d)
    out = torch.where(z > 0, out / z.clamp(min=torch.finfo(torch.float32).tiny), torch.zeros_like(out))
    lse = (m + z.log()).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, new, c["Hq"], d)[b, i]
    lse = lse.permute(0, 2, 1, 3).reshape(B, new, c["Hq"])[b, i]
    return (torch.where(have[:, None, None], out, torch.zeros_like(out)).to(torch.bfloat16),
            torch.where(have[:, None], lse, torch.full_like(lse, float("-inf"))))


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    lens, new = _lens(c)
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    if c["op"] == "append":
        starts = [sum(new[:b]) for b in range(B)]
        q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        K = torch.zeros(B, Hkv, max(new), d, dtype=torch.float64, device="cuda")
        V = torch.zeros_like(K)
        cache = s["cache"].double() if c["fmt"] == BF16 else None
        half = c["rot"] // 2
        lo = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
        hi = lo + (1 if c["interleaved"] else half)
        for b in range(B):
            rows = slice(starts[b], starts[b] + new[b])
            p = torch.arange(lens[b] - new[b], lens[b], device="cuda", dtype=torch.float64)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), p[:, None] * s["inv_freq"].double())
            both = []
            for x in (s["q"], s["k"]):
                y = x[rows].double().clone()
                w = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
                y[..., lo], y[..., hi] = w.real, w.imag
                both.append(y)
            q_out[rows] = both[0]
            v = s["v"][rows].double()
            if c["fmt"] == BF16:
                at = torch.arange(lens[b] - new[b], lens[b], device="cuda")
                pg = s["page_table"][b].long()[at // page]
                cache[pg, :, at % page, 0] = both[1]
                cache[pg, :, at % page, 1] = v
            else:
                for out, x in ((K, both[1]), (V, v)):
                    x = x.reshape(new[b], Hkv, 4, d // 4)
                    top = x.abs().amax(-1, keepdim=True) / 7
                    mant, ex = torch.frexp(top)
                    step = torch.ldexp(torch.ceil(mant * 256), ex - 8).clamp(min=1e-300)
                    out[b, :, : new[b]] = (torch.round(x / step) * step).reshape(new[b], Hkv, d).transpose(0, 1)
        return (q_out, cache) if c["fmt"] == BF16 else (q_out, K, V)
    if c["op"] == "gather":
        K = torch.zeros(B, Hkv, c["n_max"], d, dtype=torch.float64, device="cuda")
        V = torch.zeros_like(K)
        for b in range(B):
            K[b, :, : lens[b]], V[b, :, : lens[b]] = _exact_rows(s, b, lens[b])
        return K, V
    G, T = c["Hq"] // Hkv, s["q"].shape[0]
    out = torch.zeros(T, c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, c["Hq"]), float("-inf"), dtype=torch.float64, device="cuda")
    first = 0
    for b in range(B):
        n = 1 if s["seq_start"] is None else new[b]
        q = s["q"][first: first + n].double().reshape(n, Hkv, G, d)
        rows, first = slice(first, first + n), first + n
        if lens[b] == 0:
            continue
        K, V = _exact_rows(s, b, lens[b])
        for g in range(Hkv):
            keys, vals, at = K[g], V[g], torch.arange(lens[b], device="cuda")
            if c["cap"]:
                u = b * Hkv + g
                blk = s["idx"][u, : int(s["count"][u])].long()
                at = (blk[:, None] * c["unit"] + torch.arange(c["unit"], device="cuda")).flatten()
                at = at[at < lens[b]]
                keys, vals = keys[at], vals[at]
            x = torch.einsum("thd,nd->thn", q[:, g], keys) * s["sm_scale"]
            sees = at <= torch.arange(lens[b] - n, lens[b], device="cuda")[:, None]
            x = torch.where(sees[:, None], x, torch.full_like(x, float("-inf")))
            top = torch.logsumexp(x, -1)
            lse[rows, g * G: (g + 1) * G] = top
            out[rows, g * G: (g + 1) * G] = torch.einsum("thn,nd->thd", torch.exp(x - top[..., None]), vals)
    return out, lse


def _exact_rows(s, b, n):
    """Keys and values [Hkv, n, d] of sequence b in 64 bits, nibble by nibble from the format's definition."""
    c, d = s["case"], s["case"]["d"]
    at = torch.arange(n, device="cuda")
    row = s["cache"][s["page_table"][b].long()[at // c["page"]], :, at % c["page"]].transpose(0, 1)
    if c["fmt"] == BF16:
        return row[..., 0, :].double(), row[..., 1, :].double()
    K = torch.empty(c["Hkv"], n, d, dtype=torch.float64, device="cuda")
    V = torch.empty_like(K)
    sc = row[..., d:].contiguous().view(torch.bfloat16).double()
    for ch in range(d):
        g, j = divmod(ch, d // 4)
        t, e = divmod(j, d // 16)
        kb = row[..., t * (d // 8) + g * (d // 32) + e // 2].int()
        vb = row[..., d // 2 + (j % 8) * (d // 16) + g * (d // 64) + j // 16].int()
        K[..., ch] = (((kb >> 4) if e % 2 else (kb & 15)).double() - 8) * sc[..., g]
        V[..., ch] = (((vb >> 4) if j % 16 >= 8 else (vb & 15)).double() - 8) * sc[..., 4 + g]
    return K, V
