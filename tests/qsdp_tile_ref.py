"""The tiled products with coded weights in 64 bits from weights as the tiles hold them, and sizes that
reach every tile with its depth shared and not; for the tests only."""
import torch

import qsdp_linear_ref as ref

# (direction, tokens, rows, cols, tile of the plan, workgroups that share a tile's depth)
PLANNED = [
    ("linear", 149, 22787, 2592, 0, 2), ("linear", 134, 16444, 2176, 0, 3), ("linear", 8980, 136, 3168, 0, 6),
    ("linear", 133, 3137, 16256, 0, 16), ("linear", 8232, 135, 32, 1, 1), ("linear", 70, 12425, 1440, 1, 2),
    ("linear", 5776, 1, 1056, 1, 3), ("linear", 1069, 1, 1600, 1, 16), ("linear", 34, 1, 32, 2, 1),
    ("linear", 33, 11703, 2656, 2, 2), ("linear", 34, 1, 1728, 2, 16), ("linear", 34, 1, 160, 3, 1),
    ("linear", 5699, 6, 864, 3, 2), ("linear", 33, 1, 2336, 3, 12), ("linear", 34, 1, 3328, 3, 16),
    ("grad", 263, 1, 11392, 0, 1), ("grad", 4096, 6400, 1600, 0, 2), ("grad", 500, 50257, 1600, 0, 16),
    ("grad", 8239, 1886, 160, 0, 6), ("grad", 138, 5999, 2784, 0, 16), ("grad", 8330, 1, 160, 1, 1),
    ("grad", 75, 1440, 12000, 1, 2), ("grad", 66, 1081, 1504, 1, 12), ("grad", 68, 1806, 1056, 1, 16),
    ("grad", 1, 1, 32, 2, 1), ("grad", 1, 1580, 12512, 2, 2), ("grad", 1, 1565, 32, 2, 16), ("grad", 1, 130, 32, 3, 1),
    ("grad", 4229, 841, 32, 3, 2), ("grad", 709, 1030, 64, 3, 6), ("grad", 1, 3080, 32, 3, 16),
]


def tile_weights(codes, lo, hi, rows, cols, bucket, bits, dtype):
    """Weights [rows, cols] in fp64 as the tiles hold them: a fused product and sum in fp32, rounded once
    more to `dtype`.  Where a bucket's minimum and step are of like size, as in the tests' weights, code *
    delta (32 bits) and the sum are exact in fp64, so one rounding to fp32 is the fused operation's."""
    n = rows * cols
    at = torch.arange(n, device=codes.device) // bucket
    delta = ((hi - lo).double() / (2.0 ** bits - 1)).float().double()
    w = lo.double()[at] + ref.unpack(codes, bits)[:n].double() * delta[at]
    return w.float().to(dtype).double().view(rows, cols)


def tile_product(op, x, w):
    """(result in fp64, elementwise tolerance) of x [tokens, depth] with tile_weights' w [rows, cols].

    The tolerance counts the result's own rounding (half a step, of the smallest normal number at least) and
    the sums in fp32.  Let P be the largest magnitude of a sum over the first 64 k products, for any k, and
    L the largest sum of 64 products' magnitudes.  What is added up is always a stretch of whole blocks and
    part of another, so every partial sum is within 2 P + L, and a rounding to fp32 within 2^-24 of
    that.  depth + 64 of them (one for each product, the joins of groups and shares), taken as
    independent: eight times the root of their number.  (Products of values of 11 bits are exact.)"""
    if op == "linear":
        w = w.t().contiguous()
    dtype, x, depth = x.dtype, x.double(), x.shape[1]
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    most, block = torch.zeros_like(y), torch.zeros_like(y)
    for d in range(0, depth, 64):
        a, b = x[:, d:d + 64].contiguous(), w[d:d + 64]
        y = torch.addmm(y, a, b)
        most = torch.maximum(most, y.abs())
        block = torch.maximum(block, a.abs() @ b.abs())
    tol = ref.HALF_STEP[dtype] * y.abs().clamp_min(torch.finfo(dtype).tiny)
    return y, tol + 8.0 * (depth + 64) ** 0.5 * 2.0 ** -24 * (2.0 * most + block)


def coded_weights(rows, cols, bucket, bits, g, whole=False):
    """Codes, minima and maxima as the products' tests draw them.  whole: small whole weights, at most 155 in
    magnitude and exact in 8 bits of mantissa."""
    n, top = rows * cols, 2 ** bits - 1
    nb = ref.buckets(n, bucket)
    code = torch.randint(0, top + 1, (n + n % 2,), generator=g).to(torch.uint8)
    if whole:
        step = torch.ones(nb) if bits == 8 else torch.randint(1, 5, (nb,), generator=g).float()
        lo = -torch.randint(100, 129, (nb,), generator=g).float() if bits == 8 else \
            -torch.randint(0, 33, (nb,), generator=g).float()
    else:
        step = 0.02 * torch.exp(torch.randn(nb, generator=g)) / top * 8
        lo = -step * top * (0.3 + 0.4 * torch.rand(nb, generator=g))
    return ref.pack(code, bits)[:(n * bits + 7) // 8].clone(), lo, lo + step * top
