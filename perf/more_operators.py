"""Measured cases of the 8-bit path's attention: over whole prompts, of one new token over a paged
cache, and the cache's filling.

Operators: attention of packed sequences (grouped heads, causal or not, other key lengths than
query lengths); attention of one query a sequence over pages of keys and values, in 16 bits or in
E4M3 with one E8M0 scale for each key and head; and the writing of new keys and values into the
pages.  Both attentions give 16-bit rows, or, with heads of 128, codes and scales as the 8-bit
linear takes them.  Each has a plain form of elementary torch operations, the framework's call, and
its definition in 64 bits.

Sequence s has Lq queries and Lk keys; with `causal`, query i sees keys j <= i + Lk - Lq.  A query
that sees no key gives zeros.
"""

import math
import random

import torch

own = False

LARGEST = 4.0 * 128 * 32 * (8192 * 8193 // 2)   # flops of the largest listed prompt
CACHED = 2.0 * 160 * 4096 * 8 * 129             # bytes of about the largest listed cache


def listed():
    return [
        # a question of 37 tokens: latency
        dict(name="attention_short", op="attention", B=1, T=37, past="none", Hq=32, Hkv=8, D=128, causal=True,
             dtype="bf16", fp8=False, mix=1),
        # two images at the PixArt-like width (16 heads of 72) and their captions of up to 300 tokens
        dict(name="attention_caption", op="attention", B=2, T=8192, past="caption", Hq=16, Hkv=16, D=72, causal=False,
             dtype="fp16", fp8=False, mix=2),
        # the same two images' self attention
        dict(name="attention_image", op="attention", B=2, T=8192, past="none", Hq=16, Hkv=16, D=72, causal=False,
             dtype="fp16", fp8=False, mix=0),
        # 23 prompts of different lengths in one batch, narrow heads
        dict(name="attention_packed", op="attention", B=23, T=5003, past="none", Hq=16, Hkv=4, D=64, causal=True,
             dtype="fp16", fp8=False, mix=3),
        # a long prompt, codes for the output projection: the largest product
        dict(name="attention_prompt", op="attention", B=1, T=8192, past="none", Hq=32, Hkv=8, D=128, causal=True,
             dtype="bf16", fp8=True, mix=4),
        # one conversation's next token, short: latency
        dict(name="paged_token", op="paged", B=1, shortest=513, longest=513, Hq=32, Hkv=8, D=128, page=16,
             cache="bf16", dtype="bf16", fp8=False, mix=5),
        # 37 conversations of all lengths
        dict(name="paged_batch", op="paged", B=37, shortest=50, longest=4000, Hq=32, Hkv=8, D=128, page=16,
             cache="bf16", dtype="bf16", fp8=True, mix=6),
        # one key head for each query head
        dict(name="paged_heads", op="paged", B=9, shortest=1000, longest=2047, Hq=16, Hkv=16, D=64, page=32,
             cache="fp16", dtype="fp16", fp8=False, mix=7),
        # two whole books in an 8-bit cache: rows are few, the length is split
        dict(name="paged_long", op="paged", B=2, shortest=120000, longest=131072, Hq=32, Hkv=8, D=128, page=64,
             cache="fp8", dtype="bf16", fp8=False, mix=8),
        # a server's batch, 8-bit cache: the most bytes
        dict(name="paged_many", op="paged", B=160, shortest=200, longest=8000, Hq=32, Hkv=8, D=128, page=16,
             cache="fp8", dtype="fp16", fp8=True, mix=9),
        # the new tokens' keys and values of 37 conversations
        dict(name="append_tokens", op="append", B=37, T=37, shortest=50, longest=900, Hkv=8, D=128, page=16,
             cache="bf16", dtype="bf16", mix=6),
        # the keys and values of 23 prompts, 8-bit cache
        dict(name="append_prompts", op="append", B=23, T=8192, shortest=0, longest=700, Hkv=8, D=128, page=64,
             cache="fp8", dtype="bf16", mix=10),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["attention", "attention", "paged", "paged", "append"])
    Hkv, D = rng.choice([1, 2, 4, 8, 16]), rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128])
    c = dict(op=op, Hkv=Hkv, dtype=rng.choice(["bf16", "fp16"]), mix=rng.randrange(1, 1 << 30))
    if op == "attention":
        c.update(T=size(1, 8192), Hq=Hkv * rng.choice([1, 2, 4, 6, 8]), D=D, causal=rng.random() < 0.7,
                 past=rng.choice(["none", "none", "none", "longer", "caption"]), fp8=D == 128 and rng.random() < 0.5)
        c["Hq"] = Hkv * max(1, min(c["Hq"] // Hkv, 32 // Hkv))
        c["B"] = min(c["T"], size(1, 40))
        while work(c)["flops"] > LARGEST:
            c["T"] = max(c["B"], c["T"] * 3 // 4)
        return c
    c.update(B=size(1, 200), page=rng.choice([16, 32, 64, 128]), cache=rng.choice([c["dtype"], "fp8"]))
    if c["cache"] == "fp8":
        D = max(32, D // 16 * 16)
    c["D"] = D
    if op == "append":
        c.update(T=c["B"] if rng.random() < 0.5 else size(c["B"], 8192),
                 longest=max(1, min(size(16, 4000), int(1e8 / (4.0 * c["B"] * Hkv * D)))))
        c["shortest"] = rng.randrange(0, c["longest"])
        return c
    c.update(Hq=Hkv * rng.choice([1, 2, 4, 8, 16]), fp8=D == 128 and rng.random() < 0.5)
    c["longest"] = max(1, min(size(16, 131072), int(0.8 * CACHED / (2.0 * c["B"] * Hkv * D * 2))))
    c["shortest"] = rng.randrange(0, c["longest"] + 1)
    return c


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}[name]


# ------------------------------------------------------------------------- lengths

def _cut(total, parts, mix):
    """`parts` lengths of at least one that add up to `total`: equal ones for mix 0, else of all sizes."""
    if mix == 0:
        return [total // parts + (i < total % parts) for i in range(parts)]
    at = [0] + sorted(random.Random(mix).sample(range(1, total), parts - 1)) + [total]
    return [b - a for a, b in zip(at, at[1:])]


def _lengths(case):
    """Query and key lengths of each sequence (attention), cached lengths with the new tokens (paged,
    append), and the numbers of new tokens (append)."""
    r = random.Random(case["mix"] + 1)
    if case["op"] == "attention":
        q = _cut(case["T"], case["B"], case["mix"])
        if case["past"] == "none":
            return q, q
        if case["past"] == "longer":                       # a part of the prompt was there before
            return q, [n + r.randrange(0, 2 * n + 1) for n in q]
        return q, [r.randrange(20, 301) for _ in q]
    held = [r.randrange(case["shortest"], case["longest"] + 1) for _ in range(case["B"])]
    if case["op"] == "paged":
        return held, None
    new = _cut(case["T"], case["B"], case["mix"])
    return [a + b for a, b in zip(held, new)], new


def _cumulative(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------- inputs

def _heads(T, H, D, g, spread=1.0):
    """Unit Gaussian rows about a mean of their head."""
    return spread * torch.randn(T, H, D, device="cuda", generator=g) + 0.3 * torch.randn(H, D, device="cuda", generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, Hkv, D = _dtype(case["dtype"]), case["Hkv"], case["D"]
    s = dict(case=case)
    if case["op"] == "attention":
        q, k = _lengths(case)
        Hq, T = case["Hq"], sum(q)
        s["cu_q"] = s["cu_k"] = _cumulative(q)
        if case["past"] == "none":
            # views of the projection's output, as a linear of all three writes it
            qkv = torch.cat([_heads(T, Hq, D, g, 1.5), _heads(T, 2 * Hkv, D, g)], dim=1).to(dt)
            s["Q"], s["K"], s["V"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["Q"] = _heads(T, Hq, D, g, 1.5).to(dt)
            s["K"], s["V"] = _heads(sum(k), Hkv, D, g).to(dt), _heads(sum(k), Hkv, D, g).to(dt)
            s["cu_k"] = _cumulative(k)
        return s
    lengths, new = _lengths(case)
    page = case["page"]
    need = [(n + page - 1) // page for n in lengths]
    pages = sum(need) + 3
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    rows = torch.arange(max(1, max(need)), device="cuda")[None, :]
    first = _cumulative(need)[:-1, None]
    at = first + rows
    s["table"] = torch.where(rows < torch.tensor(need, device="cuda")[:, None], order[at.clamp(max=pages - 1).long()],
                             torch.full_like(at, -1)).to(torch.int32).contiguous()
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kc, vc = (_heads(pages * page, Hkv, D, g).to(dt).reshape(pages, page, Hkv, D).transpose(1, 2).contiguous()
              for _ in range(2))
    if case["cache"] == "fp8":
        (kc, s["kscales"]), (vc, s["vscales"]) = _quantize(kc), _quantize(vc)
    s["kcache"], s["vcache"] = kc, vc
    if case["op"] == "paged":
        s["Q"] = _heads(case["B"], case["Hq"], D, g, 1.5).to(dt)
        return s
    kv = _heads(case["T"], 2 * Hkv, D, g).to(dt)
    s["K"], s["V"] = kv[:, :Hkv], kv[:, Hkv:]
    s["cu"] = _cumulative(new)
    return s


# ------------------------------------------------------------------------- plain form

def _quantize(y):
    """Rows of up to 128 values -> E4M3 codes and the E8M0 byte of each row."""
    y = y.float()
    frac, ex = torch.frexp(y.abs().amax(dim=-1))             # largest = frac 2^ex, 0.5 <= frac < 1
    e = torch.where(frac <= 0.875, ex - 9, ex - 8)           # 448 = 0.875 2^9
    e = torch.where(frac > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    unit = ((127 - e) << 23).to(torch.int32).view(torch.float32)                 # 2^-e
    return (y * unit[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _padded(scales):
    """Scale bytes [T][H] as rows of whole dwords."""
    return torch.nn.functional.pad(scales, (0, -scales.shape[1] % 4))


def _as_values(codes, scales):
    return {"codes": codes, "scales": scales.view(torch.float8_e8m0fnu)}


def _values(rows, scales):
    """float32 values of cached rows."""
    rows = rows.float()
    return rows if scales is None else rows * scales.view(torch.float8_e8m0fnu).float()[..., None]


def _softmax(x, seen):
    """Weights of the visible scores and their sums; zeros and one where nothing is visible."""
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(dim=-1, keepdim=True)
    return p, torch.where(total > 0, total, torch.ones_like(total))


def _result(o, c):
    """o float32 [T][Hq][D] as the call returns it."""
    if not c["fp8"]:
        return o.to(_dtype(c["dtype"]))
    codes, scales = _quantize(o)
    return _as_values(codes.reshape(len(o), -1), _padded(scales))


def _plain_attention(s, c):
    Q, K, V, cq, ck = s["Q"], s["K"], s["V"], s["cu_q"].long(), s["cu_k"].long()
    T, Tk, Hkv, G, D = len(Q), len(K), c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    i, j = torch.arange(T, device="cuda"), torch.arange(Tk, device="cuda")
    si, sj = torch.bucketize(i, cq[1:], right=True), torch.bucketize(j, ck[1:], right=True)
    seen = si[:, None] == sj[None, :]
    if c["causal"]:
        # as seen from the sequences' ends: keys behind j at least as many as queries behind i
        seen &= (ck[1:][sj] - j)[None, :] >= (cq[1:][si] - i)[:, None]
    q = Q.float().reshape(T, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * T, D)
    x = torch.bmm(q * D ** -0.5, K.float().permute(1, 2, 0).contiguous()).reshape(Hkv, G, T, Tk)
    p, total = _softmax(x, seen)
    del x
    o = torch.bmm(p.reshape(Hkv, G * T, Tk), V.float().transpose(0, 1).contiguous())
    o = o.reshape(Hkv, G, T, D) / total
    return _result(o.permute(2, 0, 1, 3).reshape(T, Hkv * G, D), c)


def _plain_paged(s, c):
    B, Hkv, G, D, page = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["page"]
    at = s["table"].clamp(min=0).long()
    n = at.shape[1] * page

    def rows(cache, scales):                                 # [B Hkv][n][D]
        scales = None if scales is None else scales[at]
        return _values(cache[at], scales).transpose(1, 2).reshape(B * Hkv, n, D)

    k = rows(s["kcache"], s.get("kscales"))
    q = s["Q"].float().reshape(B * Hkv, G, D) * D ** -0.5
    x = torch.bmm(q, k.transpose(1, 2).contiguous()).reshape(B, Hkv * G, n)
    del k
    seen = torch.arange(n, device="cuda")[None, None, :] < s["lengths"][:, None, None]
    p, total = _softmax(x, seen)
    o = torch.bmm(p.reshape(B * Hkv, G, n), rows(s["vcache"], s.get("vscales")))
    return _result(o.reshape(B, Hkv * G, D) / total, c)


def _plain_append(s, c):
    t = torch.arange(c["T"], device="cuda")
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    at = s["lengths"].long()[b] - (s["cu"].long()[b + 1] - t)      # position in the sequence
    page, row = s["table"].long()[b, at // c["page"]], at % c["page"]
    for cache, scales, new in (("kcache", "kscales", s["K"]), ("vcache", "vscales", s["V"])):
        if c["cache"] == "fp8":
            new, byte = _quantize(new)
            s[scales][page, :, row] = byte
            s[cache].view(torch.uint8)[page, :, row] = new.view(torch.uint8)
        else:
            s[cache][page, :, row] = new


def _caches(s):
    out = dict(k=s["kcache"], v=s["vcache"])
    if "kscales" in s:
        out.update(ks=s["kscales"].view(torch.float8_e8m0fnu), vs=s["vscales"].view(torch.float8_e8m0fnu))
    return out


def run(s):
    c = s["case"]
    if own:
        import w4a4_post_quantization_amd as kq
        if c["op"] == "attention":
            out = kq.attention(s["Q"], s["K"], s["V"], s["cu_q"], s["cu_k"], causal=c["causal"], fp8=c["fp8"])
            return _as_values(*out) if c["fp8"] else out
        if c["op"] == "paged":
            out = kq.paged_attention(s["Q"], s["kcache"], s["vcache"], s["table"], s["lengths"],
                                     kscales=s.get("kscales"), vscales=s.get("vscales"), fp8=c["fp8"])
            return _as_values(*out) if c["fp8"] else out
        kq.cache_append(s["K"], s["V"], s["kcache"], s["vcache"], s["table"], s["lengths"], s["cu"],
                        kscales=s.get("kscales"), vscales=s.get("vscales"))
        return _caches(s)
    if c["op"] == "attention":
        return _plain_attention(s, c)
    if c["op"] == "paged":
        return _plain_paged(s, c)
    _plain_append(s, c)
    return _caches(s)


# ------------------------------------------------------------------------- cost and definition

def work(case):
    Hkv, D = case["Hkv"], case["D"]
    a, b = _lengths(case)
    if case["op"] == "append":
        wide = 2 * D if case["cache"] != "fp8" else D + 1
        return {"bytes": 2.0 * case["T"] * Hkv * (2 * D + wide), "flops": 2.0 * case["T"] * Hkv * D}
    Hq, rows = case["Hq"], sum(a) if case["op"] == "attention" else case["B"]
    out = rows * Hq * (2.0 * D + (D + 1 if case["fp8"] else 2 * D))
    if case["op"] == "paged":
        wide = 2 * D if case["cache"] != "fp8" else D + 1
        return {"bytes": out + 2.0 * sum(a) * Hkv * wide, "flops": 4.0 * D * Hq * sum(a)}
    pairs = 0
    for n, m in zip(a, b):
        if not case["causal"]:
            pairs += n * m
        else:                                                # query i sees min(m, i + m - n + 1) keys, if any
            f = max(0, n - m)
            pairs += (n - f) * (max(0, m - n) + 1 + m) // 2
    return {"bytes": out + 4.0 * sum(b) * Hkv * D, "flops": 4.0 * D * Hq * pairs}


def _pow2(e):
    """2^e in float64 for whole e in the normal range, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_codes(y):
    """Values of the E4M3 codes and of the scales of float64 rows, from the definition."""
    top = y.abs().max(dim=-1).values
    unit = _pow2(torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0)).clamp(min=-127.0))
    v = y / unit[..., None]
    step = _pow2(torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step, unit


def _exact_result(o, c):
    if not c["fp8"]:
        return o
    codes, unit = _exact_codes(o)
    cols = (c["Hq"] + 3) // 4 * 4
    scales = torch.full((len(o), cols), 2.0 ** -127, dtype=torch.float64, device="cuda")
    scales[:, :c["Hq"]] = unit
    return {"codes": codes.flatten(1), "scales": scales}


def _dense(rows, byte):
    return rows.double() if byte is None else rows.to(torch.float32).double() * _pow2(byte.to(torch.int64) - 127)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    Hkv, D, a = case["Hkv"], case["D"], _lengths(case)
    if case["op"] == "append":
        lengths, new = a
        out, t0 = {}, 0
        for name, byte in (("k", "kscales"), ("v", "vscales")):
            out[name] = s[name + "cache"].to(torch.float32).double()
            if byte in s:
                out[name + "s"] = _pow2(s[byte].to(torch.int64) - 127)
        table = s["table"].cpu()
        for b, (n, m) in enumerate(zip(lengths, new)):
            at = torch.arange(n - m, n)
            page, row = table[b, at // case["page"]].long().cuda(), (at % case["page"]).cuda()
            for name in ("k", "v"):
                y = s[name.upper()][t0:t0 + m].double()
                if "kscales" in s:
                    y, unit = _exact_codes(y)
                    out[name + "s"][page, :, row] = unit
                out[name][page, :, row] = y
            t0 += m
        return out
    G = case["Hq"] // Hkv
    o = torch.zeros(len(s["Q"]), case["Hq"], D, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for b in range(case["B"]):
        if case["op"] == "attention":
            n, m = a[0][b], a[1][b]
            K, V = s["K"][k0:k0 + m].double(), s["V"][k0:k0 + m].double()
            k0 += m
        else:
            n, m = 1, a[0][b]
            at = s["table"][b, :(m + case["page"] - 1) // case["page"]].long()
            K, V = (_dense(s[x + "cache"][at], s[x + "scales"][at] if x + "scales" in s else None)
                    .transpose(1, 2).reshape(-1, Hkv, D)[:m] for x in "kv")
        if m > 0:
            for h in range(case["Hq"]):
                w = torch.mm(s["Q"][q0:q0 + n, h].double(), K[:, h // G].T) / math.sqrt(D)
                if case["op"] == "attention" and case["causal"]:
                    hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
                    w[hidden] = -math.inf
                o[q0:q0 + n, h] = torch.nan_to_num(torch.softmax(w, dim=1)) @ V[:, h // G]
        q0 += n
    return _exact_result(o, case)
