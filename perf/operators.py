"""The quantized key/value cache's operators, as cases to be timed and checked.

Three operators of onebit: kvq_quantize (code rows of keys and values into a paged
cache), kvq_dequantize (read rows back), kvq_attention (attention of new tokens over
the coded cache).  `run` computes each either in its plain form (elementary torch
operations in 32 bits) or, where `own` is true, by the library's calls.

The cache: pages of `page` tokens; codes uint8 [n_pages, kv_heads, page, D*bits/8]
(4 bits: even element in the low nibble), scales fp32 [n_pages, kv_heads, page], a
pair of each for keys and values.  A row is the D values of one token and head:
code = z + rne(x * inv), inv = fl32(L / amax), scale = fl32(amax / L), L = 127 or 7,
z = 128 or 8; a value read back is (code - z) * scale.

A write case codes rows and reads the same rows back (codes are returned as the
values they stand for); a read case gathers rows of a full cache; an attend case is
one layer's attention.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one new token for each of 64 sequences in a decoding step: the smallest write
        dict(name="write_step", op="write", tokens=64, heads=8, dim=128, dtype="bf16", bits=8, page=16, run=1),
        # a long prompt entering a 4-bit cache
        dict(name="write_prompt", op="write", tokens=16384, heads=8, dim=128, dtype="bf16", bits=4, page=64, run=16384),
        # sixteen heads of 64 (the BERT-Large layout) in fp16, an odd count of rows in short runs
        dict(name="write_ragged", op="write", tokens=5003, heads=16, dim=64, dtype="f16", bits=8, page=32, run=37),
        # reading a sequence back for a consumer that needs plain rows
        dict(name="read_sequence", op="read", tokens=32768, heads=8, dim=128, dtype="bf16", bits=8, page=64, run=32768),
        # scattered single rows to fp32, wide heads, odd count
        dict(name="read_scattered", op="read", tokens=777, heads=4, dim=256, dtype="f32", bits=4, page=16, run=1),
        # one request generating: one token over a short cache (latency)
        dict(name="step_single", op="attend", batch=1, q_min=1, q_max=1, kv_min=1000, kv_max=1000, q_heads=32, heads=8,
             dim=128, dtype="bf16", bits=8, page=16, softcap=0.0, window=0, mix=1),
        # a serving step: 64 requests of very different lengths, 4-bit cache
        dict(name="step_batch", op="attend", batch=64, q_min=1, q_max=1, kv_min=100, kv_max=16000, q_heads=32, heads=8,
             dim=128, dtype="bf16", bits=4, page=64, softcap=0.0, window=0, mix=2),
        # two requests over very long caches: the work has to be split along the cache
        dict(name="step_long", op="attend", batch=2, q_min=1, q_max=1, kv_min=120000, kv_max=131072, q_heads=64,
             heads=8, dim=128, dtype="f16", bits=8, page=128, softcap=0.0, window=0, mix=3),
        # drafted tokens checked in one pass, one query head per cache head, heads of 64
        dict(name="step_drafts", op="attend", batch=24, q_min=5, q_max=5, kv_min=900, kv_max=5000, q_heads=16, heads=16,
             dim=64, dtype="bf16", bits=8, page=32, softcap=0.0, window=0, mix=4),
        # a chunk of a long prompt over what is cached: bound by matrix products
        dict(name="chunk_long", op="attend", batch=1, q_min=2048, q_max=2048, kv_min=32768, kv_max=32768, q_heads=32,
             heads=8, dim=128, dtype="bf16", bits=8, page=64, softcap=0.0, window=0, mix=5),
        # chunks and single tokens in one batch, capped scores, a sliding window, wide heads, 4-bit
        dict(name="chunk_mixed", op="attend", batch=9, q_min=1, q_max=700, kv_min=700, kv_max=9000, q_heads=16, heads=4,
             dim=256, dtype="bf16", bits=4, page=16, softcap=30.0, window=2048, mix=6),
        # a first chunk with nothing before it, fp16
        dict(name="chunk_first", op="attend", batch=3, q_min=1500, q_max=4000, kv_min=0, kv_max=0, q_heads=16, heads=16,
             dim=64, dtype="f16", bits=8, page=64, softcap=0.0, window=0, mix=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    heads = rng.choice([1, 2, 4, 5, 8, 16])
    bits = rng.choice([4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op != "attend":
        tokens = _log_int(rng, 1, 16384)
        run = rng.choice([1, _log_int(rng, 1, tokens), tokens])
        if heads * dim * tokens > 16384 * 1024:
            tokens = 16384 * 1024 // (heads * dim) - rng.randrange(100)
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, dtype=rng.choice(["bf16", "f16", "f32"]), bits=bits,
                    page=page, run=max(1, run))
    group = rng.choice([1, 1, 2, 3, 4, 8])
    q_heads = heads * group
    dtype = rng.choice(["bf16", "f16"])
    softcap = rng.choice([0.0, 0.0, 0.0, 20.0])
    window = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
    if rng.random() < 0.55:                              # single tokens or drafts
        batch = _log_int(rng, 1, 96)
        q = rng.choice([1, 1, 1, 2, 4, 7])
        top = _log_int(rng, q + 1, 100000)
        budget = 2 ** 28 // (heads * dim * batch)        # cached elements of keys, all sequences
        top = max(q + 1, min(top, budget))
        lo = rng.choice([top, max(q, top // 8)])
        q_min, q_max, kv_min, kv_max = q, q, lo, top
    else:                                                # chunks, singles among them
        batch = _log_int(rng, 1, 12)
        hi = _log_int(rng, 2, 3000)
        q_min = rng.choice([1, max(1, hi // 2)])
        top = _log_int(rng, 1, 24000)
        pairs = 2.0e9 * 128 / (dim * q_heads * batch)    # query-key pairs per head
        q_max = max(2, min(hi, int(math.sqrt(pairs))))
        q_min = min(q_min, q_max)
        kv_min, kv_max = 0, max(1, min(top, int(pairs / q_max)))
    return dict(op=op, batch=batch, q_min=q_min, q_max=q_max, kv_min=kv_min, kv_max=kv_max, q_heads=q_heads, heads=heads,
                dim=dim, dtype=dtype, bits=bits, page=page, softcap=softcap, window=window, mix=rng.randrange(10 ** 6))


def _lengths(case):
    """(q_len, kv_len) of each sequence; kv_len counts the new tokens.  Chunks sit on top
    of kv_min to kv_max cached tokens, single tokens and drafts are the last of as many."""
    r = random.Random(case["mix"])
    q_lo, q_hi, k_lo, k_hi = (case[x] for x in ("q_min", "q_max", "kv_min", "kv_max"))
    qs, ks = [], []
    for b in range(case["batch"]):
        # at least one of the longest; among chunks about one in three is a short one
        q = q_hi if b == 0 else q_lo if q_lo != q_hi and r.random() < 0.3 else r.randint(q_lo, q_hi)
        k = k_hi if b == 0 else r.randint(k_lo, k_hi)
        qs.append(q)
        ks.append(k + q if q_lo != q_hi else max(k, q))
    if q_lo != q_hi:
        both = list(zip(qs, ks))
        r.shuffle(both)
        qs, ks = [a for a, _ in both], [a for _, a in both]
    return qs, ks


def _pairs(q_len, kv_len, window):
    """(query-key pairs, keys that some query attends)"""
    first = kv_len - q_len
    if not window:
        return q_len * first + q_len * (q_len + 1) // 2, kv_len
    full = max(0, min(q_len, kv_len - max(first, window - 1)))      # queries with a whole window
    short = q_len - full
    return full * window + short * first + short * (short + 1) // 2, min(kv_len, q_len + window - 1)


def work(case):
    row = case["dim"] * case["bits"] // 8 + 4
    if case["op"] != "attend":
        n = 2 * case["tokens"] * case["heads"]
        plain = n * case["dim"] * _BYTES[case["dtype"]]
        if case["op"] == "read":
            return {"bytes": n * row + plain + 8 * case["tokens"], "flops": n * case["dim"]}
        # written and read back: input, codes out, codes in, output
        return {"bytes": 2 * n * row + 2 * plain + 16 * case["tokens"], "flops": 4 * n * case["dim"]}
    pairs = keys = pages = new = 0
    for q, k in zip(*_lengths(case)):
        p, a = _pairs(q, k, case["window"])
        pairs, keys, new = pairs + p, keys + a, new + q
        pages += -(-a // case["page"])
    io = 2 * new * case["q_heads"] * case["dim"] * 2
    return {"bytes": io + 2 * keys * case["heads"] * row + 4 * pages + 8 * case["batch"],
            "flops": 4 * case["dim"] * pairs * case["q_heads"]}


# ------------------------------------------------------------------ inputs

def _levels(bits):
    return (127.0, 128) if bits == 8 else (7.0, 8)


def _code_rows(x, bits):
    """Codes (uint8, one a value) and scales of fp32 rows x [..., D]."""
    top, z = _levels(bits)
    amax = x.abs().amax(-1)
    live = amax >= 2.0 ** -110
    # in fp64: a division by or of a Python number multiplies by a reciprocal, two roundings in fp32
    inv = torch.where(live, (top / amax.double()).float(), torch.zeros_like(amax))
    # the product of two fp32 numbers is exact in fp64, and round() takes ties to even
    code = (x.double() * inv.double().unsqueeze(-1)).round() + z
    return code.to(torch.uint8), torch.where(live, (amax.double() / top).float(), torch.zeros_like(amax))


def _pack(code, bits):
    return code if bits == 8 else code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(packed, bits):
    if bits == 8:
        return packed
    return torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


def _slots(n, page, run, n_pages, gen, r):
    """Cache positions of n tokens: runs of consecutive tokens, each run in pages of its own."""
    order = torch.randperm(n_pages, generator=gen).tolist()
    out, used = [], 0
    while len(out) < n:
        m = min(run, n - len(out))
        start = r.randrange(page) if run < n else 0
        for i in range(start // page, (start + m - 1) // page + 1):
            lo, hi = max(start, i * page), min(start + m, (i + 1) * page)
            base = order[used] * page
            out.extend(range(base + lo - i * page, base + hi - i * page))
            used += 1
    return torch.tensor(out, dtype=torch.int64)


def _rows(gen, shape, dtype):
    """Key or value rows: normal values with a spread between channels and a few far ones."""
    d = shape[-1]
    spread = 0.5 + torch.rand(shape[-2], d, generator=gen, device="cuda")
    spread[:, :: max(1, d // 3)] *= 4.0
    return (torch.randn(shape, generator=gen, device="cuda") * spread).to(dtype)


def _fill(codes, scales, gen, bits, dim):
    """A cache filled with coded random rows, some pages at a time."""
    n_pages, heads, page = scales.shape
    step = max(1, (1 << 25) // (heads * page * dim))
    for a in range(0, n_pages, step):
        b = min(n_pages, a + step)
        x = _rows(gen, ((b - a) * page, heads, dim), torch.bfloat16).float().view(b - a, page, heads, dim)
        code, scale = _code_rows(x.transpose(1, 2).contiguous(), bits)
        codes[a:b] = _pack(code, bits)
        scales[a:b] = scale


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dim, heads, bits, page = case["dim"], case["heads"], case["bits"], case["page"]
    dt = _DT[case["dtype"]]
    s = {"case": case, "bits": bits, "page": page, "dim": dim, "heads": heads, "dtype": dt}

    def cache(n_pages):
        s["n_pages"] = n_pages
        for x in "kv":
            s[x + "_codes"] = torch.zeros(n_pages, heads, page, dim * bits // 8, dtype=torch.uint8, device="cuda")
            s[x + "_scales"] = torch.zeros(n_pages, heads, page, dtype=torch.float32, device="cuda")

    if case["op"] != "attend":
        n, run = case["tokens"], case["run"]
        need = -(-n // run) * (-(-run // page) + 1) + 3
        cache(need)
        s["slots"] = _slots(n, page, run, need, host, r).cuda()
        s["k_out"] = torch.empty(n, heads, dim, dtype=dt, device="cuda")
        s["v_out"] = torch.empty(n, heads, dim, dtype=dt, device="cuda")
        if case["op"] == "write":
            # keys and values as a projection leaves them: one row of both for each token
            kv = torch.empty(n, 2 * heads, dim, dtype=dt, device="cuda")
            kv[:, :heads] = _rows(gen, (n, heads, dim), dt)
            kv[:, heads:] = _rows(gen, (n, heads, dim), dt)
            s["k"], s["v"] = kv[:, :heads], kv[:, heads:]
        else:
            for x in "kv":
                _fill(s[x + "_codes"], s[x + "_scales"], gen, bits, dim)
        return s

    qs, ks = _lengths(case)
    hq = case["q_heads"]
    need = [-(-k // page) for k in ks]
    cache(sum(need) + 3)
    for x in "kv":
        _fill(s[x + "_codes"], s[x + "_scales"], gen, bits, dim)
    order = torch.randperm(s["n_pages"], generator=host)
    table = torch.zeros(len(qs), max(need), dtype=torch.int32)
    used = 0
    for b, m in enumerate(need):
        table[b, :m] = order[used:used + m].int()
        used += m
    offsets = [0]
    for q in qs:
        offsets.append(offsets[-1] + q)
    s["q_lens"], s["kv_host"], s["offsets"] = qs, ks, offsets
    s["table"] = table.cuda()
    s["kv_lens"] = torch.tensor(ks, dtype=torch.int32).cuda()
    # queries as a fused projection leaves them: the keys and values of the new tokens beside them
    qkv = torch.randn(offsets[-1], hq + 2 * heads, dim, generator=gen, device="cuda").to(dt)
    s["q"] = qkv[:, :hq]
    s["scale"] = 1.0 / math.sqrt(dim)
    s["out"] = torch.empty(offsets[-1], hq, dim, dtype=dt, device="cuda")
    # every sequence with as many new tokens: no offsets are needed
    s["q_offsets"] = None if min(qs) == max(qs) else torch.tensor(offsets, dtype=torch.int32).cuda()
    if own:
        from error_compensated_bit_amd import onebit
        size = onebit.kvq_attention_workspace_bytes(len(qs), offsets[-1], hq, heads, dim)
        s["workspace"] = torch.zeros(size // 8, dtype=torch.int64, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        from error_compensated_bit_amd import onebit as ob
        pools = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        if op == "attend":
            ob.kvq_attention(s["q"], *pools, s["table"], s["kv_lens"], s["out"], bits=s["bits"], scale=s["scale"],
                             q_offsets=s["q_offsets"], softcap=s["case"]["softcap"], window=s["case"]["window"],
                             workspace=s["workspace"])
            return s["out"]
        if op == "write":
            ob.kvq_quantize(s["k"], s["v"], s["slots"], *pools, bits=s["bits"])
        ob.kvq_dequantize(*pools, s["slots"], s["k_out"], s["v_out"], bits=s["bits"])
        return s["k_out"], s["v_out"]
    if op == "attend":
        return _attend(s)
    page, z = s["page"], _levels(s["bits"])[1]
    at, off = s["slots"] // page, s["slots"] % page
    outs = []
    for x in "kv":
        codes, scales = s[x + "_codes"], s[x + "_scales"]
        if op == "write":
            code, scale = _code_rows(s[x].float(), s["bits"])
            codes[at, :, off] = _pack(code, s["bits"])
            scales[at, :, off] = scale
        y = (_unpack(codes[at, :, off], s["bits"]).float() - z) * scales[at, :, off].unsqueeze(-1)
        outs.append(y.to(s["dtype"]))
    return tuple(outs)


def _attend(s):
    case, page, dim, heads, hq = s["case"], s["page"], s["dim"], s["heads"], s["case"]["q_heads"]
    z, group = _levels(s["bits"])[1], hq // heads
    out = torch.empty(s["offsets"][-1], hq, dim, dtype=s["dtype"], device="cuda")
    for b, (m, n) in enumerate(zip(s["q_lens"], s["kv_host"])):
        first, a = n - m, s["offsets"][b]
        pages = s["table"][b, :-(-n // page)].long()
        k, v = ((_unpack(s[x + "_codes"][pages], s["bits"]).float() - z) * s[x + "_scales"][pages].unsqueeze(-1)
                for x in "kv")                                          # [pages, heads, page, dim]
        k, v = (t.transpose(0, 1).reshape(heads, -1, dim)[:, :n] for t in (k, v))
        q = s["q"][a:a + m].float().view(m, heads, group, dim).permute(1, 2, 0, 3).reshape(heads, group * m, dim)
        pos = first + torch.arange(m, device="cuda").unsqueeze(1)
        key = torch.arange(n, device="cuda").unsqueeze(0)
        out_of = key > pos
        if case["window"]:
            out_of = out_of | (key <= pos - case["window"])
        out_of = out_of.repeat(group, 1)
        # a few heads at a time, so that the scores fit
        step = max(1, min(heads, (1 << 30) // max(1, group * m * n)))
        for h in range(0, heads, step):
            e = min(heads, h + step)
            x = torch.matmul(q[h:e], k[h:e].transpose(1, 2).contiguous()) * s["scale"]
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            x = x.masked_fill(out_of, -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            y = torch.matmul(x, v[h:e]) / x.sum(-1, keepdim=True)       # [heads, group * m, dim]
            y = y.view(e - h, group, m, dim).permute(2, 0, 1, 3).reshape(m, (e - h) * group, dim)
            out[a:a + m, h * group:e * group] = y.to(s["dtype"])
    return out


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    top, z = (127.0, 128.0) if case["bits"] == 8 else (7.0, 8.0)

    def value(codes, scales):
        if case["bits"] == 4:
            both = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device="cuda")
            both[..., 0::2] = (codes % 16).double()
            both[..., 1::2] = (codes // 16).double()
        else:
            both = codes.double()
        return (both - z) * scales.double()[..., None]

    if case["op"] == "write":
        outs = []
        for x in (s["k"], s["v"]):
            x = x.double()
            peak = x.abs().max(-1, keepdim=True)[0]
            # the scale and its reciprocal are held in fp32; nothing else is rounded
            inv = (top / peak).float().double()
            inv[peak < 2.0 ** -110] = 0.0
            scale = (peak / top).float().double()
            outs.append(torch.round(x * inv) * scale)
        return tuple(outs)
    if case["op"] == "read":
        flat = s["slots"]
        outs = []
        for x in "kv":
            pages, inside = flat.div(case["page"], rounding_mode="floor"), flat.remainder(case["page"])
            outs.append(value(s[x + "_codes"][pages, :, inside], s[x + "_scales"][pages, :, inside]))
        return tuple(outs)

    total = sum(s["q_lens"])
    out = torch.zeros(total, case["q_heads"], case["dim"], dtype=torch.float64, device="cuda")
    per = case["q_heads"] // case["heads"]
    row = 0
    for b in range(case["batch"]):
        m, n = s["q_lens"][b], s["kv_host"][b]
        token = torch.arange(n, device="cuda")
        page_of = s["table"][b].long()[token // case["page"]]
        for g in range(case["heads"]):
            k = value(s["k_codes"][page_of, g, token % case["page"]], s["k_scales"][page_of, g, token % case["page"]])
            v = value(s["v_codes"][page_of, g, token % case["page"]], s["v_scales"][page_of, g, token % case["page"]])
            kt = k.t().contiguous()
            for h in range(g * per, (g + 1) * per):
                for lo in range(0, m, 4096):
                    hi = min(m, lo + 4096)
                    x = (s["q"][row + lo:row + hi, h].double() @ kt) / math.sqrt(case["dim"])
                    if case["softcap"]:
                        x = torch.tanh(x / case["softcap"]) * case["softcap"]
                    p = torch.arange(n - m + lo, n - m + hi, device="cuda")[:, None]
                    keep = token[None, :] <= p
                    if case["window"]:
                        keep &= token[None, :] > p - case["window"]
                    x[~keep] = -math.inf
                    out[row + lo:row + hi, h] = torch.softmax(x, -1) @ v
        row += m
    return out
