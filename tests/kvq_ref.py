"""The coded key/value cache in 64 bits: plain CPU code written from the formulas of
include/onebit.h, for the tests only."""
import math

import numpy as np
import torch

LEVELS = {4: (7.0, 8), 8: (127.0, 128)}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def largest_scale(bits):
    """The largest fp32 number whose product with L does not exceed fp32's range."""
    biggest = np.finfo(np.float32).max
    c = np.float32(float(biggest) / LEVELS[bits][0])
    return float(c if float(c) * LEVELS[bits][0] <= float(biggest) else np.nextafter(c, np.float32(0)))


def code_rows(x, bits):
    """(codes uint8 [..., D], scales fp32 [...]) of rows x (any float type)."""
    top, z = LEVELS[bits]
    x = x.double()
    amax = x.abs().amax(-1)                       # NaN where the row holds one
    finite = torch.isfinite(amax)
    live = finite & (amax >= 2.0 ** -110)
    safe = torch.where(live, amax, torch.ones_like(amax))
    # a quotient of two 24-bit numbers rounded to 53 and then to 24 bits is the correctly rounded one
    inv, scale = (torch.full_like(safe, top) / safe).float(), (safe / torch.full_like(safe, top)).float()
    scale = scale.clamp_max(largest_scale(bits))
    code = (torch.where(live.unsqueeze(-1), x, torch.zeros_like(x)) * inv.double().unsqueeze(-1)).round() + z
    scale = torch.where(live, scale, torch.zeros_like(scale))
    return code.to(torch.uint8), torch.where(finite, scale, torch.full_like(scale, math.nan))


def pack(code, bits):
    return code if bits == 8 else code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(packed, bits):
    return packed if bits == 8 else torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


def values(packed, scales, bits):
    """Values in fp64 before any rounding."""
    return (unpack(packed, bits).double() - LEVELS[bits][1]) * scales.double().unsqueeze(-1)


def attention(q, pools, table, kv_lens, *, bits, scale, q_offsets=None, softcap=0.0, window=0):
    """(out, lse, tol, lse_tol, owned): fp64 outputs, the elementwise tolerance for an output before
    its own rounding and for lse, and which rows belong to a sequence.  All arguments on the CPU.

    The tolerance counts, per row and output element, with A = sum_j softmax_j |v_j|:
      - the weights' rounding to fp16, 2^-11 of each term: 2^-11 A (their sum and the rounded
        terms' own weights cancel no better than that);
      - the scores: D products and their sum in fp32 and a few scalings.  The sum is of codes, as
        exact as if each were 1024 (8 bits) or 64 (4 bits) in place of c - z, that is R = 1024 or 64
        scales in place of k_d: (D + 8) 2^-24 R scale_j sum_d |q_d| each.  exp2's argument is
        rounded at the size of the score itself and exp2 is good to an ulp: 2^-22 (|s| + 1); a
        capped score is off by 2^-21 cap, and for caps above 64 by 2^-21 of the score itself below an
        eighth of the cap (so by 2^-18 |s| at most).  An error e of every score moves each weight and their sum
        by e: 2 e A;
      - the sums over n terms in fp32, of codes too: (n + 64) 2^-24 (A + R sum_j softmax_j scale_j),
        twice.
    Chunks (more than 48 rows, tokens x heads of a cache head) of bf16 take the rows as fp16: the
    scale and the product are each rounded once, 2^-10 of a key or value, and what fp16's range cuts
    off is below 2^-14 of the largest scale: 2^-10 sum_d |q_d k_d| + 2^-14 max(scale) sum_d |q_d| for
    a score, 2^-10 A + 2^-14 max(scale) for an output.
    Weights far below the row's largest lose bits to fp16's range: 2^-31 of the largest
    scale's row for each of the n terms.  lse is off by what the scores are, the sum's n roundings
    and its own (2^-22 of its size).
    """
    k_codes, k_scales, v_codes, v_scales = pools
    n_pages, heads, page, _ = k_codes.shape
    total, hq, dim = q.shape
    group = hq // heads
    batch, max_pages = table.shape
    top, reach = LEVELS[bits][0], {8: 1024.0, 4: 64.0}[bits]
    out = torch.zeros(total, hq, dim, dtype=torch.float64)
    tol = torch.zeros(total, hq, dim, dtype=torch.float64)
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros(total, hq, dtype=torch.float64)
    owned = torch.zeros(total, dtype=torch.bool)
    offs = [b * (total // batch) for b in range(batch + 1)] if q_offsets is None else q_offsets.tolist()
    for b in range(batch):
        lo, hi = offs[b], offs[b + 1]
        m, n = hi - lo, min(max(int(kv_lens[b]), 0), max_pages * page)
        owned[lo:hi] = True
        if not m or not n:
            continue
        at = torch.arange(n)
        pages = table[b].long()[at // page]
        there = (pages >= 0) & (pages < n_pages)
        pages = pages.clamp(0, n_pages - 1)
        pos = n - m + torch.arange(m).unsqueeze(1)
        keep = (at <= pos) & there
        if window:
            keep &= at > pos - window
        used = keep.any(0)
        for g in range(heads):
            ks, vs = k_scales[pages, g, at % page], v_scales[pages, g, at % page]
            # what nobody attends to has no influence, whatever it holds
            ks, vs = (torch.where(used, s, torch.zeros_like(s)) for s in (ks, vs))
            k = values(k_codes[pages, g, at % page], ks, bits)
            v = values(v_codes[pages, g, at % page], vs, bits)
            for h in range(g * group, (g + 1) * group):
                x = q[lo:hi, h].double()
                s = scale * (x @ k.T)
                size = abs(scale) * reach * x.abs().sum(1, keepdim=True) * ks.double().abs()
                off = (dim + 8) * 2.0 ** -24 * size + 2.0 ** -22 * (s.abs() + 1)
                rounded = q.dtype == torch.bfloat16 and m * group > 48
                k_top, v_top = (float(torch.nan_to_num(t, posinf=0.0).abs().max()) for t in (ks, vs))
                if rounded:
                    off = off + abs(scale) * (2.0 ** -10 * (x.abs() @ k.abs().T) +
                                              2.0 ** -14 * k_top * x.abs().sum(1, keepdim=True))
                if softcap:
                    off = off + 2.0 ** -21 * (softcap if softcap <= 64 else (8 * s.abs()).clamp(max=softcap))
                    s = softcap * torch.tanh(s / softcap)
                s = s.masked_fill(~keep, -math.inf)
                some = keep.any(1)
                peak = torch.where(some, s.amax(1), torch.zeros(m, dtype=torch.float64))
                e = torch.exp(s - peak.unsqueeze(1)).masked_fill(~keep, 0.0)
                l = e.sum(1)
                p = e / torch.where(some, l, torch.ones_like(l)).unsqueeze(1)
                # a value is left out by its mask, not by a weight of 0: a kept NaN stays one
                out[lo:hi, h] = p @ v
                lse[lo:hi, h] = torch.where(some, peak + torch.log(l), torch.full_like(l, -math.inf))
                worst = torch.where(keep, off, torch.zeros_like(off)).amax(1, keepdim=True)
                count = keep.sum(1, keepdim=True).double()
                a = p @ v.abs()
                lse_tol[lo:hi, h] = (worst + (count + 64) * 2.0 ** -24).squeeze(1) + 2.0 ** -22 * (lse[lo:hi, h].abs() + 1)
                wide = a + reach * (p @ vs.double().abs()).unsqueeze(1)
                tol[lo:hi, h] = a * (2.0 ** -11 + 2 * worst) + 2 * (count + 64) * 2.0 ** -24 * wide + \
                    count * 2.0 ** -31 * v_top * top + (2.0 ** -10 * a + 2.0 ** -14 * v_top if rounded else 0.0)
    return out, lse, tol, lse_tol, owned
