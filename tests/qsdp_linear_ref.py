"""Products with coded weights in 64 bits: plain CPU code written from the formulas of
include/onebit.h, for the tests only."""
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def pack(code, bits):
    return code if bits == 8 else code[0::2] | (code[1::2] << 4)


def unpack(packed, bits):
    return packed if bits == 8 else torch.stack((packed & 15, packed >> 4), -1).flatten()


def buckets(n, bucket):
    return -(-n // bucket)


def weights(codes, lo, hi, rows, cols, bucket, bits):
    """(w [rows, cols], delta of each of them) in fp64; delta is held in fp32."""
    n = rows * cols
    at = torch.arange(n) // bucket
    # a quotient of two 24-bit numbers rounded to 53 and then to 24 bits is the correctly rounded one
    delta = ((hi - lo).double() / (2.0 ** bits - 1)).float().double()
    w = lo.double()[at] + unpack(codes, bits)[:n].double() * delta[at]
    return w.view(rows, cols), delta[at].view(rows, cols)


def product(x, w, delta, bits, dtype, exact):
    """(result in fp64, elementwise tolerance) of x [tokens, depth] times w [depth, width].

    The tolerance counts, with A = sum |x| |w|, S = sum |x|:
      - the result's own rounding: half a step of the result (of the smallest normal number at least);
      - `exact` false: each weight's rounding to the type, half a step of it each: half a step of A.
        (No less: a bucket has 2^bits different weights, so the errors of equal codes are equal and do not
        average out.  With one bucket a row, 130 of 2080 weights share one error, and where x has a mean of
        half its spread their sum is 130 / 2 spreads and not sqrt(130).)  Weights of fp16 below 2^-14
        are off by 2^-25;
      - the sums in fp32.  Where codes and minima enter apart (`exact`), a code stands for at most
        R = 32 (4 bits, an offset of 16 in front) or 256 (8 bits) steps of its bucket, so terms and
        partial sums are within B = A + R sum |x| delta, else within A.  depth + 64 roundings of 2^-24,
        taken as independent: eight times the root of their number.
    """
    x, a = x.double(), x.double().abs()
    y = x @ w
    half = HALF_STEP[dtype]
    big = a @ w.abs()
    tol = half * y.abs().clamp_min(torch.finfo(dtype).tiny)
    if exact:
        big = big + (32.0 if bits == 4 else 256.0) * (a @ delta)
    else:
        tol = tol + half * big
        if dtype == torch.float16:
            tol = tol + 2.0 ** -25 * a.sum(1, keepdim=True)
    return y, tol + 8.0 * (x.shape[1] + 64) ** 0.5 * 2.0 ** -24 * big
