"""Products with coded weights and the rotating append to the coded cache, as cases to be timed and checked.

Three operators of onebit: qsdp_linear (rows times a matrix kept in qsdp_quantize's
codes), qsdp_linear_grad (the gradient of its input, from the same codes) and kvq_append
(queries and keys turned by their positions, keys and values coded into the paged cache).
`run` computes each either in its plain form (elementary torch operations in 32 bits) or,
where `own` is true, by the library's calls.

A matrix [n_out, n_in] is the flat vector of its rows, coded by buckets of `bucket`
values: w = min + code * delta, delta = (max - min) / (2^bits - 1), codes of 4 bits two a
byte, the even value in the low nibble.  `linear`: out[t, o] = sum_i x[t, i] w[o, i];
`grad`: dx[t, i] = sum_o dy[t, o] w[o, i].

`append`: the first `rot` values of a query or key head are pairs, (i, i + rot / 2) or
(2 i, 2 i + 1), turned by the angle of their position and index, whose cosine and sine
stand in a table [positions, rot]; keys and values are then coded as kvq_quantize does:
code = z + rne(x * inv), inv = fl32(L / amax), scale = fl32(amax / L), L = 127 or 7,
z = 128 or 8, and read back from the cache as (code - z) * scale.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one request's next token through a feed-forward matrix, buckets that run across rows
        dict(name="linear_single", op="linear", tokens=1, n_in=1600, n_out=6400, dtype="bf16", bits=4, bucket=1024),
        # a decoding step of 32 requests through a wide layer
        dict(name="linear_batch", op="linear", tokens=32, n_in=8192, n_out=28672, dtype="bf16", bits=4, bucket=128),
        # drafted tokens scored over a vocabulary of odd size, 8 bits
        dict(name="linear_head", op="linear", tokens=5, n_in=1600, n_out=50257, dtype="f16", bits=8, bucket=1024),
        # a short prompt, fine groups
        dict(name="linear_short", op="linear", tokens=77, n_in=4096, n_out=4096, dtype="f16", bits=4, bucket=64),
        # an odd number of tokens through a fused projection
        dict(name="linear_ragged", op="linear", tokens=333, n_in=1600, n_out=4800, dtype="f16", bits=8, bucket=1024),
        # a long prompt: bound by matrix products
        dict(name="linear_prompt", op="linear", tokens=2048, n_in=4096, n_out=16384, dtype="bf16", bits=4, bucket=256),
        # a few tokens' gradient, the finest groups
        dict(name="grad_short", op="grad", tokens=19, n_in=1024, n_out=4096, dtype="bf16", bits=4, bucket=32),
        # a training batch through a feed-forward matrix
        dict(name="grad_batch", op="grad", tokens=4096, n_in=1600, n_out=6400, dtype="bf16", bits=4, bucket=1024),
        # the loss's gradient through a vocabulary of odd size
        dict(name="grad_head", op="grad", tokens=500, n_in=1600, n_out=50257, dtype="f16", bits=8, bucket=1024),
        # one new token for each of 64 sequences
        dict(name="append_step", op="append", tokens=64, q_heads=32, heads=8, dim=128, rot=128, pairs="halves",
             dtype="bf16", bits=8, page=16, run=1, far=32768),
        # a long prompt entering a 4-bit cache
        dict(name="append_prompt", op="append", tokens=16384, q_heads=32, heads=8, dim=128, rot=128, pairs="halves",
             dtype="bf16", bits=4, page=64, run=16384, far=131072),
        # short runs of many sequences, neighbouring values as pairs, half of a head turned
        dict(name="append_ragged", op="append", tokens=5003, q_heads=16, heads=16, dim=64, rot=32, pairs="neighbours",
             dtype="f16", bits=8, page=32, run=37, far=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "grad", "grad", "append"])
    bits = rng.choice([4, 8])
    if op == "append":
        dim = rng.choice([64, 128, 128, 256])
        heads = rng.choice([1, 2, 4, 5, 8, 16])
        q_heads = heads * rng.choice([1, 2, 3, 4, 8])
        dtype = rng.choice(["bf16", "f16", "f32"])
        most = 16384 * 6144 * 2 // ((q_heads + 2 * heads) * dim * _BYTES[dtype])
        tokens = max(1, min(_log_int(rng, 1, 16384), most - rng.randrange(9)))
        run = rng.choice([1, _log_int(rng, 1, tokens), tokens])
        return dict(op=op, tokens=tokens, q_heads=q_heads, heads=heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 16 * rng.randint(1, dim // 16)]),
                    pairs=rng.choice(["halves", "neighbours"]), dtype=dtype, bits=bits,
                    page=rng.choice([16, 32, 64, 128]), run=run, far=_log_int(rng, max(run, 512), 131072))
    n_in = 32 * _log_int(rng, 2, 256)
    n_out = _log_int(rng, 48, 60000)
    n_out = min(n_out, 2 ** 27 // n_in)
    top = int(1.3e11 / (n_in * n_out))                   # tokens within the largest case's products
    tokens = max(1, min(_log_int(rng, 1, 4096), top))
    bucket = rng.choice([32, 64, 128, 128, 256, 1024, 1024, 32 * rng.randint(1, 64), n_in])
    return dict(op=op, tokens=tokens, n_in=n_in, n_out=n_out, dtype=rng.choice(["bf16", "f16"]), bits=bits,
                bucket=bucket)


def work(case):
    t = case["tokens"]
    if case["op"] != "append":
        n = case["n_in"] * case["n_out"]
        weights = n * case["bits"] // 8 + 8 * -(-n // case["bucket"])
        return {"bytes": weights + 2 * t * (case["n_in"] + case["n_out"]), "flops": 2 * t * n}
    dim, heads, size = case["dim"], case["heads"], _BYTES[case["dtype"]]
    row = dim * case["bits"] // 8 + 4
    q = t * case["q_heads"] * dim
    kv = 2 * t * heads
    # queries in and out, keys and values in, codes written and read back, the rows read back, table, slots, positions
    return {"bytes": 2 * q * size + 2 * kv * dim * size + 2 * kv * row + t * (4 * case["rot"] + 24),
            "flops": 6 * t * (case["q_heads"] + heads) * case["rot"] // 2 + 4 * kv * dim}


# ------------------------------------------------------------------ inputs

def _pack(code, bits):
    return code if bits == 8 else code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(packed, bits):
    if bits == 8:
        return packed
    return torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


def _coded_weights(case, gen):
    """Codes, minima and maxima of normal weights, some rows and some single ones larger."""
    n_in, n_out, bits, bucket = case["n_in"], case["n_out"], case["bits"], case["bucket"]
    n, top = n_in * n_out, 2 ** bits - 1
    w = torch.randn(n_out, n_in, generator=gen, device="cuda").mul_(0.02)
    w *= 0.5 + torch.rand(n_out, 1, generator=gen, device="cuda")
    w.view(-1)[:: 4999] *= 4.0
    w = w.bfloat16().float().view(-1)
    pad = -n % bucket
    if pad:
        w = torch.cat((w, w[-1:].expand(pad)))
    w = w.view(-1, bucket)
    lo, hi = w.amin(1), w.amax(1)
    t = (w - lo.unsqueeze(1)) / ((hi - lo) / top).clamp_min(1e-30).unsqueeze(1)
    code = (t + torch.rand(t.shape, generator=gen, device="cuda")).floor_().clamp_(0, top).to(torch.uint8)
    return _pack(code.view(-1)[:n], bits).contiguous(), lo, hi


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, tokens, bits = _DT[case["dtype"]], case["tokens"], case["bits"]
    s = {"case": case, "bits": bits, "dtype": dt}
    if case["op"] != "append":
        n_in, n_out = case["n_in"], case["n_out"]
        s["codes"], s["lo"], s["hi"] = _coded_weights(case, gen)
        a, b = (n_in, n_out) if case["op"] == "linear" else (n_out, n_in)
        # rows start on 16 bytes, so a vocabulary of odd size has padded rows
        pad = torch.full((tokens, a + -a % 8), math.nan, dtype=dt, device="cuda")
        s["x"] = pad[:, :a]
        if case["op"] == "linear":
            # activations behind a norm: normal values, a few channels far larger
            x = torch.randn(tokens, a, generator=gen, device="cuda")
            x[:, :: 97] *= 8.0
        else:
            # gradients: tokens of very different weight
            x = torch.randn(tokens, a, generator=gen, device="cuda") * 1e-2
            x *= torch.exp(torch.randn(tokens, 1, generator=gen, device="cuda"))
        s["x"].copy_(x)
        s["out"] = torch.empty(tokens, b, dtype=dt, device="cuda")
        if own:
            from error_compensated_bit_amd import onebit
            size = onebit.qsdp_linear_workspace_bytes(tokens, n_out, n_in)
            s["workspace"] = torch.zeros(max(1, size // 8), dtype=torch.int64, device="cuda")
        return s

    host = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    dim, heads, hq, page, run = case["dim"], case["heads"], case["q_heads"], case["page"], case["run"]
    need = -(-tokens // run) * (-(-run // page) + 1) + 3
    s["page"] = page
    for x in "kv":
        s[x + "_codes"] = torch.zeros(need, heads, page, dim * bits // 8, dtype=torch.uint8, device="cuda")
        s[x + "_scales"] = torch.zeros(need, heads, page, dtype=torch.float32, device="cuda")
    s["slots"] = _slots(tokens, page, run, need, host, r).cuda()
    # every run of tokens starts somewhere in its sequence
    first = torch.randint(0, max(1, case["far"] - run + 1), (-(-tokens // run),), generator=host)
    s["positions"] = (first.repeat_interleave(run)[:tokens] + torch.arange(tokens) % run).cuda()
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(case["far"], dtype=torch.float64, device="cuda").unsqueeze(1) * freq
    s["rotary"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    # queries, keys and values as a projection leaves them: one row of all three for each token
    qkv = torch.randn(tokens, hq + 2 * heads, dim, generator=gen, device="cuda")
    qkv *= 0.5 + torch.rand(hq + 2 * heads, dim, generator=gen, device="cuda")
    qkv = qkv.to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
    s["q_out"] = torch.empty(tokens, hq, dim, dtype=dt, device="cuda")
    s["k_out"] = torch.empty(tokens, heads, dim, dtype=dt, device="cuda")
    s["v_out"] = torch.empty(tokens, heads, dim, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from error_compensated_bit_amd import onebit as ob
        if op != "append":
            call = ob.qsdp_linear if op == "linear" else ob.qsdp_linear_grad
            call(s["x"], s["codes"], s["lo"], s["hi"], s["out"], bucket=case["bucket"], bits=s["bits"],
                 workspace=s["workspace"])
            return s["out"]
        pools = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        ob.kvq_append(s["q"], s["k"], s["v"], s["positions"], s["rotary"], s["slots"], *pools, s["q_out"],
                      bits=s["bits"], interleaved=case["pairs"] == "neighbours")
        ob.kvq_dequantize(*pools, s["slots"], s["k_out"], s["v_out"], bits=s["bits"])
        return s["q_out"], s["k_out"], s["v_out"]
    if op == "append":
        return _append(s)
    w = _weights(s)
    return torch.matmul(s["x"].float(), w.t() if op == "linear" else w).to(s["dtype"])


def _weights(s):
    case, top = s["case"], 2 ** s["bits"] - 1
    n, bucket = case["n_in"] * case["n_out"], case["bucket"]
    code = _unpack(s["codes"], s["bits"]).float()
    if n % bucket:
        code = torch.cat((code, code.new_zeros(bucket - n % bucket)))
    w = s["lo"].unsqueeze(1) + code.view(-1, bucket) * ((s["hi"] - s["lo"]) / top).unsqueeze(1)
    return w.view(-1)[:n].view(case["n_out"], case["n_in"])


def _turn(x, table, rot, neighbours):
    """The first `rot` values of each row turned: products of fp32 numbers are exact in fp64, and their
    difference or sum is rounded to fp32 at the end."""
    half = rot // 2
    c, d = table[:, None, :half].double(), table[:, None, half:].double()
    y = x.float().double()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if neighbours else (y[..., :half], y[..., half:rot])
    p, q = a * c - b * d, b * c + a * d
    turned = torch.stack((p, q), -1).flatten(-2) if neighbours else torch.cat((p, q), -1)
    return torch.cat((turned, y[..., rot:]), -1).float()


def _append(s):
    case, page, z = s["case"], s["page"], _levels(s["bits"])[1]
    table = s["rotary"][s["positions"]]
    at, off = s["slots"] // page, s["slots"] % page
    neighbours = case["pairs"] == "neighbours"
    outs = [_turn(s["q"], table, case["rot"], neighbours).to(s["dtype"])]
    for x in "kv":
        rows = _turn(s["k"], table, case["rot"], neighbours) if x == "k" else s["v"].float()
        codes, scales = s[x + "_codes"], s[x + "_scales"]
        code, scale = _code_rows(rows, s["bits"])
        codes[at, :, off] = _pack(code, s["bits"])
        scales[at, :, off] = scale
        y = (_unpack(codes[at, :, off], s["bits"]).float() - z) * scales[at, :, off].unsqueeze(-1)
        outs.append(y.to(s["dtype"]))
    return tuple(outs)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "append":
        n_in, n_out, bucket = case["n_in"], case["n_out"], case["bucket"]
        at = torch.arange(n_in * n_out, device="cuda")
        if case["bits"] == 4:
            byte = s["codes"][at // 2]
            code = torch.where(at % 2 == 0, byte % 16, byte // 16).double()
        else:
            code = s["codes"].double()
        at //= bucket
        step = (s["hi"].double() - s["lo"].double()) / (2.0 ** case["bits"] - 1.0)
        w = (code * step[at] + s["lo"].double()[at]).reshape(n_out, n_in)
        x = s["x"].double()
        return x @ (w.t().contiguous() if case["op"] == "linear" else w)

    top, rot = (127.0 if case["bits"] == 8 else 7.0), case["rot"]
    i = torch.arange(case["dim"], device="cuda")
    if case["pairs"] == "neighbours":
        other, index, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0).double()
    else:
        low = i < rot // 2
        other, index, sign = torch.where(low, i + rot // 2, i - rot // 2), i % (rot // 2), torch.where(low, -1.0, 1.0).double()
    turned = i < rot
    other, index = torch.where(turned, other, i), torch.where(turned, index, 0)
    cos = s["rotary"].double()[s["positions"]][:, index]
    sin = s["rotary"].double()[s["positions"]][:, index + rot // 2] * sign
    cos, sin = torch.where(turned, cos, 1.0)[:, None], torch.where(turned, sin, 0.0)[:, None]
    outs = []
    for x in "qkv":
        y = s[x].double()
        if x != "v":
            y = y * cos + y[..., other] * sin
        if x == "q":
            outs.append(y)
            continue
        # rows are held in fp32 before they are coded, their scale and its reciprocal too
        y = y.float().double()
        peak = y.abs().max(-1, keepdim=True)[0]
        inv = (top / peak).float().double()
        inv[peak < 2.0 ** -110] = 0.0
        outs.append(torch.round(y * inv) * (peak / top).float().double())
    return tuple(outs)
