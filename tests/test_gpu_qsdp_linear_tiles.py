"""The tiled products with coded weights on the GPU, every tile with its depth shared and not: whole numbers
to the bit, others within a tolerance that sees a step left out (qsdp_tile_ref.tile_product)."""
import math

import pytest
import torch

import qsdp_tile_ref as tiles
from test_gpu_qsdp_linear import BF16, DEV, F16, dev, gen, padded, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op,tokens,rows,cols,shape,splits", tiles.PLANNED)
@pytest.mark.parametrize("bits,bucket,dtype", [(4, 1024, BF16), (8, 96, F16)])
def test_every_tile_to_the_bit(op, tokens, rows, cols, shape, splits, bits, bucket, dtype):
    """Inputs of -2 .. 2, whole weights up to 155, depths up to 50257: every partial sum is below 2^24 and
    so exact, and a result is the exact one rounded once, whatever the order."""
    depth = cols if op == "linear" else rows
    assert depth * 2 * 155 < 2 ** 24
    g = gen("tiles", op, rows, cols, bits)
    weights = dev(tiles.coded_weights(rows, cols, bucket, bits, g, whole=True))
    x = torch.randint(-2, 3, (tokens, depth), generator=g).to(dtype)
    w = tiles.tile_weights(*weights, rows, cols, bucket, bits, dtype)
    want = (x.to(DEV).double() @ (w.t().contiguous() if op == "linear" else w)).float().to(dtype)
    got = run(op, padded(x), weights, rows, cols, bucket, bits)
    assert torch.equal(got, want), float((got.float() - want.float()).abs().max())


@pytest.mark.parametrize("op,tokens,rows,cols,shape,splits", tiles.PLANNED)
@pytest.mark.parametrize("bits,bucket,dtype", [(4, 96, F16), (8, 1024, BF16)])
def test_every_tile_within_its_sums_roundings(op, tokens, rows, cols, shape, splits, bits, bucket, dtype):
    g = gen("sums", op, rows, cols, bits)
    weights = dev(tiles.coded_weights(rows, cols, bucket, bits, g))
    x = torch.randn(tokens, cols if op == "linear" else rows, generator=g).to(dtype)
    w = tiles.tile_weights(*weights, rows, cols, bucket, bits, dtype)
    want, tol = tiles.tile_product(op, x.to(DEV), w)
    off = (run(op, padded(x), weights, rows, cols, bucket, bits).double() - want).abs() / tol
    assert torch.all(off <= 1.0), float(off.max())


@pytest.mark.parametrize("op,rows,cols", [("linear", 333, 160), ("linear", 1000, 2080), ("grad", 333, 160), ("grad", 2081, 1024)])
@pytest.mark.parametrize("tokens", [33, 64, 129, 515])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_products_within_their_sums_roundings(op, rows, cols, tokens, bits, dtype):
    """Inputs with a mean, tokens of very different size, buckets across rows."""
    bucket = 1088
    g = gen("means", op, rows, cols, tokens)
    weights = dev(tiles.coded_weights(rows, cols, bucket, bits, g))
    x = torch.randn(tokens, cols if op == "linear" else rows, generator=g)
    x = (x * torch.exp(torch.randn(tokens, 1, generator=g)) + 0.5 * torch.randn(tokens, 1, generator=g)).to(dtype)
    w = tiles.tile_weights(*weights, rows, cols, bucket, bits, dtype)
    want, tol = tiles.tile_product(op, x.to(DEV), w)
    off = (run(op, padded(x), weights, rows, cols, bucket, bits).double() - want).abs() / tol
    assert torch.all(off <= 1.0), float(off.max())


def test_shared_depths_repeat_to_the_bit_and_no_token_sees_another():
    """The largest tile with its depth shared by 16, a workspace that holds anything before."""
    op, tokens, rows, cols = next(p[:4] for p in tiles.PLANNED if p[0] == "grad" and p[4:] == (0, 16))
    bucket, bits = 1024, 4
    g = gen("repeat tiles")
    weights = dev(tiles.coded_weights(rows, cols, bucket, bits, g))
    x = torch.randn(tokens, rows, generator=g).to(BF16)
    one = run(op, padded(x), weights, rows, cols, bucket, bits)
    assert torch.equal(one, run(op, padded(x), weights, rows, cols, bucket, bits))
    x[7] = math.inf
    two = run(op, padded(x), weights, rows, cols, bucket, bits)
    others = [t for t in range(tokens) if t != 7]
    assert torch.equal(one[others], two[others]) and not torch.any(torch.isfinite(two[7]))
