"""The tiled products with coded weights on the GPU, every tile with its depth shared and not: whole numbers
to the bit."""
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
