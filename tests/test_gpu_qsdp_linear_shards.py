"""Products with weights that ranks quantized shard by shard and gathered."""
import pytest
import torch

import qsdp_linear_ref as ref
from error_compensated_bit_amd import onebit as ob
from test_gpu_qsdp_linear import BF16, DEV, EXACT, gen, run

pytestmark = pytest.mark.gpu


def quantized(x, bucket, bits, seed):
    n = x.numel()
    codes = torch.zeros((n * bits + 7) // 8, dtype=torch.uint8, device=DEV)
    lo, hi = (torch.zeros(ref.buckets(n, bucket), device=DEV) for _ in range(2))
    ob.qsdp_quantize(x, bucket, bits, seed, codes, lo, hi)
    return codes, lo, hi


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,cols,cuts,bucket", [
    (96, 160, (5120, 10240), 1024),            # shards that end inside rows
    (96, 160, (4800, 9600), 32),               # whole rows, the finest buckets
    (50, 96, (1536, 2880), 96),                # a short last shard
])
def test_gathered_shards(bits, rows, cols, cuts, bucket):
    g = gen("shards", rows, bits)
    w = (torch.randn(rows * cols, generator=g) * 0.02).to(BF16).to(DEV)
    parts = [p.clone() for p in torch.tensor_split(w, cuts)]
    assert all(p.numel() % bucket == 0 for p in parts[:-1])
    coded = [quantized(p, bucket, bits, 5 + i) for i, p in enumerate(parts)]
    # every shard decoded by itself
    decoded = torch.cat([ref.weights(*(t.cpu() for t in c), 1, p.numel(), bucket, bits)[0].flatten()
                         for c, p in zip(coded, parts)]).view(rows, cols)
    delta = torch.cat([ref.weights(*(t.cpu() for t in c), 1, p.numel(), bucket, bits)[1].flatten()
                       for c, p in zip(coded, parts)]).view(rows, cols)
    whole = [torch.cat(t) for t in zip(*coded)]
    for op, tokens in (("linear", 5), ("linear", 70), ("grad", 5), ("grad", 70)):
        x = torch.randn(tokens, cols if op == "linear" else -(-rows // 8) * 8, generator=g).to(BF16)[:, :cols if op == "linear" else rows]
        a, d = (decoded.t().contiguous(), delta.t().contiguous()) if op == "linear" else (decoded, delta)
        want, tol = ref.product(x, a, d, bits, BF16, op == "linear" and tokens <= EXACT)
        xd = torch.zeros(tokens, -(-x.shape[1] // 8) * 8, dtype=BF16, device=DEV)
        xd[:, :x.shape[1]] = x.to(DEV)
        got = run(op, xd[:, :x.shape[1]], whole, rows, cols, bucket, bits).cpu().double()
        assert torch.all((got - want).abs() <= tol), (op, tokens)


def test_shards_that_end_inside_buckets_are_matrices_of_their_own():
    """Two shards of 35 rows of 96 in buckets of 1024 have four buckets each; one matrix of them has seven and
    is refused for their number."""
    g = gen("apart")
    w = (torch.randn(70 * 96, generator=g) * 0.02).to(BF16).to(DEV)
    x = torch.randn(3, 96, generator=g).to(BF16)
    coded = [quantized(p.clone(), 1024, 8, 3) for p in w.view(2, -1)]
    out = torch.zeros(3, 70, dtype=BF16, device=DEV)
    for c, o in zip(coded, (out[:, :35], out[:, 35:])):
        a, d = (t.t().contiguous() for t in ref.weights(*(t.cpu() for t in c), 35, 96, 1024, 8))
        run("linear", x.to(DEV), c, 35, 96, 1024, 8, out=o)
        want, tol = ref.product(x, a, d, 8, BF16, True)
        assert torch.all((o.cpu().double() - want).abs() <= tol)
    with pytest.raises(ValueError):
        run("linear", x.to(DEV), [torch.cat(t) for t in zip(*coded)], 70, 96, 1024, 8)
