"""Weights outside fp16's range: what the products with coded weights document for them."""
import math

import pytest
import torch

import qsdp_linear_ref as ref
import qsdp_tile_ref as tiles
from test_gpu_qsdp_linear import BF16, DEV, EXACT, F16, dev, gen, padded, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["linear", "grad"])
@pytest.mark.parametrize("tokens", [1, EXACT, EXACT + 1, 200])
@pytest.mark.parametrize("bits", [4, 8])
def test_weights_above_65504(op, tokens, bits):
    """One bucket reaches 131040: its weights of 65520 or more are infinite where weights are rounded to fp16 and
    themselves where codes enter apart, and for bf16 everywhere."""
    rows, cols, bucket = 90, 160, 160
    g = gen("range", op, tokens, bits)
    codes, lo, hi = tiles.coded_weights(rows, cols, bucket, bits, g)
    hit, top = 40, 2 ** bits - 1
    lo[hit], hi[hit] = 0.0, 131040.0        # steps of 8736 (4 bits; 7 of them are 61152) or 513.88
    code = ref.unpack(codes, bits).view(rows, cols)
    x = torch.randn(tokens, cols if op == "linear" else rows, generator=g) * 2.0 ** -14
    for dtype in (F16, BF16):
        xt = x.to(dtype)
        got = run(op, padded(xt), dev((codes, lo, hi)), rows, cols, bucket, bits).cpu().double()
        w, delta = ref.weights(codes, lo, hi, rows, cols, bucket, bits)
        exact = op == "linear" and tokens <= EXACT
        if op == "linear":
            over = torch.zeros(rows, dtype=torch.bool)
            over[hit] = True
            w, delta = w.t(), delta.t()
        else:
            over = code[hit].double() * (131040.0 / top) >= 65520.0
        want, tol = ref.product(xt, w.contiguous(), delta.contiguous(), bits, dtype, exact)
        if dtype == F16 and not exact:
            assert over.any() and not torch.any(torch.isfinite(got[:, over]))
        else:
            over = torch.zeros_like(over)
        assert torch.all((got - want).abs()[:, ~over] <= tol[:, ~over])
