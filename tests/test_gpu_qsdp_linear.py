"""Products with coded weights on the GPU: results that are whole numbers to the bit, others within
tolerances that count roundings (qsdp_linear_ref.product)."""
import math
import zlib

import pytest
import torch

import qsdp_linear_ref as ref
from error_compensated_bit_amd import onebit as ob

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16
EXACT = ob.QSDP_LINEAR_EXACT_TOKENS
CALL = {"linear": ob.qsdp_linear, "grad": ob.qsdp_linear_grad}


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def coded(rows, cols, bucket, bits, g, whole=False):
    """Codes, minima and maxima.  whole: small whole weights, exact in 8 bits of mantissa."""
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


def run(op, x, weights, rows, cols, bucket, bits, workspace=None, out=None, stream=None):
    tokens = x.shape[0]
    width = rows if op == "linear" else cols
    if out is None:
        out = torch.full((tokens, width), math.nan, dtype=x.dtype, device=DEV)
    if workspace is None:
        # what it holds before does not matter
        workspace = torch.full((ob.qsdp_linear_workspace_bytes(tokens, rows, cols),), 0xFF, dtype=torch.uint8, device=DEV)
    CALL[op](x, *weights, out, bucket=bucket, bits=bits, workspace=workspace, stream=stream)
    return out


def expect(op, x, weights, rows, cols, bucket, bits, tokens=None):
    """(fp64 result, tolerance) on the GPU (fp64 products, whatever the size)."""
    w, delta = ref.weights(*[t.cpu() for t in weights], rows, cols, bucket, bits)
    w, delta = w.to(DEV), delta.to(DEV)
    if op == "linear":
        w, delta = w.t().contiguous(), delta.t().contiguous()
    exact = op == "linear" and (x.shape[0] if tokens is None else tokens) <= EXACT
    return ref.product(x, w, delta, bits, x.dtype, exact)


def dev(ts):
    return tuple(t.to(DEV) for t in ts)


def padded(x):
    """x as rows that start on 16 bytes, NaN between them."""
    t, n = x.shape
    y = torch.full((t, n + -n % 8 + 8), math.nan, dtype=x.dtype, device=DEV)
    y[:, :n] = x.to(DEV)
    return y[:, :n]


TOKENS = [1, 2, 15, 16, 17, 32, 33, 48, 63, 64, 65, 100, 129, 300]
# (rows, cols, bucket): single rows, odd counts, buckets inside, across and over many rows
SHAPES = [(1, 32, 32), (17, 32, 1024), (40, 64, 32), (127, 160, 1024), (200, 96, 96), (65, 416, 64), (33, 1600, 1024),
          (300, 128, 128), (129, 1024, 256), (50, 2080, 2080), (260, 544, 1088), (16, 4096, 65536)]


@pytest.mark.parametrize("op", ["linear", "grad"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,cols,bucket", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_whole_numbers_come_out_to_the_bit(op, bits, rows, cols, bucket, dtype):
    """Inputs of -2 .. 2, whole weights up to 155: every product and sum is exact in fp32, so a result
    is the exact one rounded once, whatever the order."""
    for tokens in TOKENS:
        g = gen("whole", op, rows, cols, tokens)
        weights = coded(rows, cols, bucket, bits, g, whole=True)
        x = torch.randint(-2, 3, (tokens, cols if op == "linear" else rows), generator=g).to(dtype)
        # fp16's range ends at 65504
        want = expect(op, x.to(DEV), weights, rows, cols, bucket, bits)[0].float().to(dtype)
        got = run(op, padded(x), dev(weights), rows, cols, bucket, bits)
        assert torch.equal(got, want), (tokens, (got.float() - want.float()).abs().max())


@pytest.mark.parametrize("op", ["linear", "grad"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,cols,bucket", SHAPES + [(6400, 1600, 1024), (515, 8192, 128), (5003, 64, 32)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_products_within_the_counted_roundings(op, bits, rows, cols, bucket, dtype):
    for tokens in (1, 3, 16, 32, 33, 64, 65, 200, 515):
        g = gen("product", op, rows, cols, tokens)
        weights = coded(rows, cols, bucket, bits, g)
        x = torch.randn(tokens, cols if op == "linear" else rows, generator=g)
        x = (x * torch.exp(torch.randn(tokens, 1, generator=g)) + 0.5 * torch.randn(tokens, 1, generator=g)).to(dtype)
        want, tol = expect(op, x.to(DEV), weights, rows, cols, bucket, bits)
        got = run(op, padded(x), dev(weights), rows, cols, bucket, bits)
        off = (got.double() - want).abs() / tol
        assert torch.all(off <= 1.0), (tokens, float(off.max()))


@pytest.mark.parametrize("op,rows,cols", [("linear", 3333, 160), ("linear", 3400, 1600), ("grad", 133, 3360), ("grad", 1601, 3392)])
@pytest.mark.parametrize("bits,bucket", [(4, 1024), (4, 32), (8, 96), (8, 1600)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_tokens(op, rows, cols, bits, bucket, dtype):
    """Products with enough tiles for the largest ones, whole numbers and others."""
    tokens = 4100
    g = gen("many", op, rows, bits)
    depth = cols if op == "linear" else rows
    weights = coded(rows, cols, bucket, bits, g, whole=True)
    x = torch.randint(-2, 3, (tokens, depth), generator=g).to(dtype)
    want = expect(op, x.to(DEV), weights, rows, cols, bucket, bits)[0].float().to(dtype)
    assert torch.equal(run(op, padded(x), dev(weights), rows, cols, bucket, bits), want)
    weights = coded(rows, cols, bucket, bits, g)
    x = torch.randn(tokens, depth, generator=g).to(dtype)
    want, tol = expect(op, x.to(DEV), weights, rows, cols, bucket, bits)
    assert torch.all((run(op, padded(x), dev(weights), rows, cols, bucket, bits).double() - want).abs() <= tol)


@pytest.mark.parametrize("bits,bucket", [(4, 128), (8, 1024)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,cols", [(16500, 256), (16411, 4224)])
def test_large_matrices(rows, cols, bits, bucket, dtype):
    """Up to 64 tokens over matrices of enough rows and columns for the widest streams."""
    g = gen("large", rows, bits)
    weights = dev(coded(rows, cols, bucket, bits, g, whole=True))
    for tokens in (1, 16, 17, 32, 33, 50, 64, 65):
        x = torch.randint(-2, 3, (tokens, cols), generator=g).to(dtype)
        want = expect("linear", x.to(DEV), weights, rows, cols, bucket, bits)[0].float().to(dtype)
        assert torch.equal(run("linear", padded(x), weights, rows, cols, bucket, bits), want), tokens


# each number of the matrix's rows that a workgroup of the streaming kernel takes, with one bucket of a row's
# 128 columns and with several; rows that end inside a workgroup's
@pytest.mark.parametrize("rows,cols", [(4095, 640), (4097, 384), (8193, 384), (9000, 1120), (20001, 256), (32771, 128),
                                       (32800, 1440)])
@pytest.mark.parametrize("bits,bucket", [(4, 128), (4, 96), (8, 256), (8, 1024)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_few_tokens_times_many_rows(rows, cols, bits, bucket, dtype):
    for tokens in (1, 16, 17, 32):
        g = gen("few", rows, cols, bits, bucket, tokens)
        weights = coded(rows, cols, bucket, bits, g)
        x = torch.randn(tokens, cols, generator=g).to(dtype)
        want, tol = expect("linear", x.to(DEV), weights, rows, cols, bucket, bits)
        got = run("linear", padded(x), dev(weights), rows, cols, bucket, bits)
        off = (got.double() - want).abs() / tol
        assert torch.all(off <= 1.0), (tokens, float(off.max()))


@pytest.mark.parametrize("tokens", [5, 40, 130])
@pytest.mark.parametrize("bits", [4, 8])
def test_gradient_is_the_products_differences(tokens, bits):
    """out is linear in x: <dy, f(x + e d) - f(x - e d)> / 2 e = <dx, d>, in whole numbers throughout."""
    rows, cols, bucket = 70, 96, 1024
    g = gen("difference", tokens, bits)
    weights = dev(coded(rows, cols, bucket, bits, g, whole=True))
    x, d = (torch.randint(-1, 2, (tokens, cols), generator=g).to(BF16).to(DEV) for _ in range(2))
    dy = torch.randint(-1, 2, (tokens, rows), generator=g).to(BF16).to(DEV)
    dx = run("grad", padded(dy), weights, rows, cols, bucket, bits)
    # of columns one at a time, so that a difference is a weight itself and exact in bf16
    for i in (0, 31, 32, 95):
        e = torch.zeros_like(x)
        e[:, i] = 1
        up, down = (run("linear", e * s, weights, rows, cols, bucket, bits) for s in (1, -1))
        slope = ((up.double() - down.double()) / 2 * dy.double()).sum(1)
        assert torch.equal(slope.float().to(BF16), dx[:, i]), i


@pytest.mark.parametrize("op", ["linear", "grad"])
@pytest.mark.parametrize("tokens", [1, 30, 64, 65, 300])
def test_strides_offsets_and_what_is_left_alone(op, tokens):
    """Rows inside wider buffers: what is between rows and behind the last stays, also with odd strides."""
    rows, cols, bucket, bits = 131, 160, 1024, 4
    a, b = (cols, rows) if op == "linear" else (rows, cols)
    g = gen("strides", op, tokens)
    weights = dev(coded(rows, cols, bucket, bits, g, whole=True))
    x = torch.randint(-2, 3, (tokens, a), generator=g).to(BF16)
    want = expect(op, x.to(DEV), weights, rows, cols, bucket, bits)[0].float().to(BF16)
    wide = torch.full((tokens + 2, a + -a % 8 + 40), math.nan, dtype=BF16, device=DEV)
    wide[1:tokens + 1, 16:16 + a] = x.to(DEV)
    for width, first in ((b, 0), (b + 1, 1), (b + 7, 3), (b + 64, 8)):
        out = torch.full((tokens + 2, width + 3), 7.0, dtype=BF16, device=DEV)
        run(op, wide[1:tokens + 1, 16:16 + a], weights, rows, cols, bucket, bits, out=out[1:tokens + 1, first:first + b])
        assert torch.equal(out[1:tokens + 1, first:first + b], want)
        left = torch.ones_like(out, dtype=torch.bool)
        left[1:tokens + 1, first:first + b] = False
        assert torch.all(out[left] == 7.0)


@pytest.mark.parametrize("op", ["linear", "grad"])
@pytest.mark.parametrize("tokens", [3, 64, 100])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_finite_stays_where_it_belongs(op, tokens, bits, dtype, bad):
    rows, cols, bucket = 90, 160, 96
    a, b = (cols, rows) if op == "linear" else (rows, cols)
    g = gen("bad", op, tokens, bits)
    clean = coded(rows, cols, bucket, bits, g)
    x = torch.randn(tokens, a, generator=g).to(dtype)
    base = run(op, x.to(DEV) if a % 8 == 0 else padded(x), dev(clean), rows, cols, bucket, bits)
    # one value of one token
    y = x.clone()
    y[tokens - 2, a - 1] = bad
    got = run(op, padded(y), dev(clean), rows, cols, bucket, bits)
    others = [t for t in range(tokens) if t != tokens - 2]
    assert torch.equal(got[others], base[others])
    assert not torch.any(torch.isfinite(got[tokens - 2]))
    # one bucket's minimum (which its maximum then shares), then its maximum alone
    hit = (torch.arange(rows * cols) // bucket == 40).view(rows, cols)
    hit = hit.any(1 if op == "linear" else 0)
    for which in ((1, 2), (2,), (1,)):
        weights = [t.clone() for t in clean]
        for k in which:
            weights[k][40] = bad
        got = run(op, padded(x), dev(weights), rows, cols, bucket, bits).cpu()
        assert torch.equal(got[:, ~hit], base.cpu()[:, ~hit]), which
        assert not torch.any(torch.isfinite(got[:, hit])), which


@pytest.mark.parametrize("op", ["linear", "grad"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_constant_and_zero_buckets(op, dtype):
    """A bucket whose values are all equal has steps of 0: its weights are its minimum."""
    rows, cols, bucket, bits = 64, 64, 64, 4
    g = gen("constant", op)
    codes, lo, hi = coded(rows, cols, bucket, bits, g, whole=True)
    hi[::2] = lo[::2]
    lo[::4] = hi[::4] = 0.0
    for tokens in (2, 64, 90):
        x = torch.randint(-2, 3, (tokens, 64), generator=g).to(dtype).to(DEV)
        want = expect(op, x, (codes, lo, hi), rows, cols, bucket, bits)[0].float().to(dtype)
        assert torch.equal(run(op, x, dev((codes, lo, hi)), rows, cols, bucket, bits), want)


@pytest.mark.parametrize("op", ["linear", "grad"])
def test_weights_of_very_different_size(op):
    """Buckets from 2^-20 to 2^8: each result by its own tolerance."""
    rows, cols, bucket, bits = 150, 256, 32, 8
    g = gen("sizes", op)
    codes, lo, hi = coded(rows, cols, bucket, bits, g)
    f = torch.exp2(torch.randint(-20, 9, lo.shape, generator=g).float())
    lo, hi = lo * f, hi * f
    for tokens in (7, 64, 77):
        for dtype in (BF16, F16):
            x = torch.randn(tokens, cols if op == "linear" else rows, generator=g).to(dtype)
            want, tol = expect(op, x.to(DEV), (codes, lo, hi), rows, cols, bucket, bits)
            got = run(op, padded(x), dev((codes, lo, hi)), rows, cols, bucket, bits)
            assert torch.all((got.double() - want).abs() <= tol)


@pytest.mark.parametrize("op", ["linear", "grad"])
@pytest.mark.parametrize("tokens", [4, 64, 200])
def test_results_repeat_to_the_bit_and_no_token_sees_another(op, tokens):
    rows, cols, bucket, bits = 700, 1600, 1024, 4
    g = gen("repeat", op, tokens)
    weights = dev(coded(rows, cols, bucket, bits, g))
    a = cols if op == "linear" else rows
    x = torch.randn(tokens, a, generator=g).to(BF16)
    one = run(op, padded(x), weights, rows, cols, bucket, bits)
    assert torch.equal(one, run(op, padded(x), weights, rows, cols, bucket, bits))
    x[0] = 1e30
    two = run(op, padded(x), weights, rows, cols, bucket, bits)
    assert torch.equal(one[1:], two[1:])


@pytest.mark.parametrize("op", ["linear", "grad"])
def test_no_tokens_and_an_own_stream(op):
    rows, cols, bucket, bits = 90, 96, 32, 8
    g = gen("stream", op)
    weights = dev(coded(rows, cols, bucket, bits, g, whole=True))
    a, b = (cols, rows) if op == "linear" else (rows, cols)
    assert run(op, torch.zeros(0, a, dtype=F16, device=DEV), weights, rows, cols, bucket, bits).shape == (0, b)
    side = torch.cuda.Stream()
    x = torch.randint(-2, 3, (120, a), generator=g).to(F16)
    xd = padded(x)
    want = expect(op, x.to(DEV), weights, rows, cols, bucket, bits)[0].float().to(F16)
    ws = torch.zeros(ob.qsdp_linear_workspace_bytes(120, rows, cols), dtype=torch.uint8, device=DEV)
    out = torch.zeros(120, b, dtype=F16, device=DEV)
    torch.cuda.synchronize()
    run(op, xd, weights, rows, cols, bucket, bits, workspace=ws, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.stream(side):
        out2 = run(op, xd, weights, rows, cols, bucket, bits, workspace=ws)
    side.synchronize()
    assert torch.equal(out2, want)


@pytest.mark.parametrize("tokens", [2, 90])
def test_captured_and_replayed(tokens):
    """Forward and gradient in one graph, replayed with new inputs and eager work in between."""
    rows, cols, bucket, bits = 640, 1600, 1024, 4
    g = gen("graph", tokens)
    weights = dev(coded(rows, cols, bucket, bits, g))
    x = torch.randn(tokens, cols, generator=g).to(BF16).to(DEV)
    out, dx = torch.zeros(tokens, rows, dtype=BF16, device=DEV), torch.zeros(tokens, cols, dtype=BF16, device=DEV)
    ws = torch.zeros(ob.qsdp_linear_workspace_bytes(tokens, rows, cols), dtype=torch.uint8, device=DEV)
    eager_ws = torch.zeros_like(ws)

    def both(o, d, w):
        run("linear", x, weights, rows, cols, bucket, bits, workspace=w, out=o)
        run("grad", o, weights, rows, cols, bucket, bits, workspace=w, out=d)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(out, dx, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(out, dx, ws)
    for _ in range(4):
        x.copy_(torch.randn(tokens, cols, generator=g))
        want = torch.zeros_like(out), torch.zeros_like(dx)
        both(*want, eager_ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(dx, want[1])


def test_two_calls_at_once():
    """Two streams with a workspace each, tiles whose depth is shared."""
    rows, cols, bucket, bits, tokens = 500, 4096, 1024, 4, 90
    g = gen("two")
    weights = dev(coded(rows, cols, bucket, bits, g, whole=True))
    xs = [torch.randint(-2, 3, (tokens, cols), generator=g).to(BF16) for _ in range(2)]
    want = [expect("linear", x.to(DEV), weights, rows, cols, bucket, bits)[0].float().to(BF16) for x in xs]
    xd = [padded(x) for x in xs]
    ws = [torch.zeros(ob.qsdp_linear_workspace_bytes(tokens, rows, cols), dtype=torch.uint8, device=DEV) for _ in xs]
    outs = [[torch.zeros(tokens, rows, dtype=BF16, device=DEV) for _ in range(8)] for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for i in range(8):
        for k in range(2):
            run("linear", xd[k], weights, rows, cols, bucket, bits, workspace=ws[k], out=outs[k][i], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, want[k]) for o in outs[k])


@pytest.mark.parametrize("tokens", [2, 40])
def test_codes_past_4_gib(tokens):
    """A matrix of 5.4e9 weights, 5 GiB of codes: rows far apart, by single columns and single rows."""
    rows, cols, bucket, bits = 1 << 20, 5120, 1024, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.randint(0, 256, (rows * cols,), generator=g, dtype=torch.uint8, device=DEV)
    lo = -torch.randint(100, 129, (rows * cols // bucket,), generator=g, device=DEV).float()
    hi = lo + 255.0
    look = torch.tensor([0, 1, 77777, 409600, 419430, 838860, 838861, rows - 2, rows - 1], device=DEV)
    flat = look.unsqueeze(1) * cols + torch.arange(cols, device=DEV)
    w = lo[flat // bucket] + codes[flat].float()                            # whole numbers up to 155
    x = torch.zeros(tokens, cols, dtype=BF16, device=DEV)
    x[0, 5], x[1, 5119], x[1, 7] = 1, 1, 1
    ws = torch.zeros(ob.qsdp_linear_workspace_bytes(tokens, rows, cols), dtype=torch.uint8, device=DEV)
    out = torch.zeros(tokens, rows, dtype=BF16, device=DEV)
    ob.qsdp_linear(x, codes, lo, hi, out, bucket=bucket, bits=bits, workspace=ws)
    assert torch.equal(out[:, look].float(), (x.float() @ w.t()).to(BF16).float())
    dy = torch.zeros(tokens, rows, dtype=BF16, device=DEV)
    for i, r in enumerate(look.tolist()):
        dy[i % tokens, r] = 1
    dx = torch.zeros(tokens, cols, dtype=BF16, device=DEV)
    ob.qsdp_linear_grad(dy, codes, lo, hi, dx, bucket=bucket, bits=bits, workspace=ws)
    assert torch.equal(dx.float(), (dy[:, look].float() @ w).to(BF16).float())


def test_rows_of_the_input_far_apart():
    """Strides near their limit: a tile's rows span more than 2 GiB."""
    rows, cols, bucket, bits, tokens, stride = 96, 128, 128, 4, 260, (1 << 23) - 8
    g = gen("far rows")
    weights = dev(coded(rows, cols, bucket, bits, g, whole=True))
    room = torch.empty(tokens * stride, dtype=BF16, device=DEV)
    for op, a in (("linear", cols), ("grad", rows)):
        x = torch.randint(-2, 3, (tokens, a), generator=g).to(BF16).to(DEV)
        far = room.view(tokens, stride)[:, 16:16 + a]
        far.copy_(x)
        want = expect(op, x, weights, rows, cols, bucket, bits)[0].float().to(BF16)
        assert torch.equal(run(op, far, weights, rows, cols, bucket, bits), want)
        assert torch.equal(run(op, far[:20], weights, rows, cols, bucket, bits), want[:20])


def test_bindings_refusals():
    rows, cols, bucket, bits = 96, 64, 128, 4
    weights = dev(coded(rows, cols, bucket, bits, gen("refuse")))
    x, out = torch.zeros(3, cols, dtype=BF16, device=DEV), torch.zeros(3, rows, dtype=BF16, device=DEV)
    ws = torch.zeros(ob.qsdp_linear_workspace_bytes(3, rows, cols), dtype=torch.uint8, device=DEV)

    def call(x=x, codes=weights[0], lo=weights[1], hi=weights[2], out=out, bucket=bucket, bits=bits, ws=ws):
        ob.qsdp_linear(x, codes, lo, hi, out, bucket=bucket, bits=bits, workspace=ws)

    call()
    for error, kw in [(ValueError, dict(out=out.half())), (ValueError, dict(out=out[:2])), (ValueError, dict(bits=3)),
                      (ValueError, dict(bits=8)), (ValueError, dict(bucket=0)), (ValueError, dict(bucket=64)),
                      (ValueError, dict(codes=weights[0][1:])), (ValueError, dict(lo=weights[1][:-1])),
                      (ValueError, dict(hi=weights[2][:-1])), (TypeError, dict(codes=weights[0].view(torch.int8))),
                      (TypeError, dict(lo=weights[1].double())), (ValueError, dict(x=x.t().contiguous().t())),
                      (ValueError, dict(x=x[0])), (TypeError, dict(x=x.cpu())), (TypeError, dict(ws=ws.cpu())),
                      (ValueError, dict(ws=torch.zeros(64, 64, device=DEV).t())),
                      (ob.OnebitError, dict(x=x.float(), out=out.float())), (ob.OnebitError, dict(ws=ws[:0])),
                      (ob.OnebitError, dict(x=torch.zeros(3, 68, dtype=BF16, device=DEV)[:, :64])),
                      (ob.OnebitError, dict(x=torch.zeros(200, dtype=BF16, device=DEV)[4:196].view(3, 64))),
                      (ob.OnebitError, dict(x=x[:1].expand(3, cols)))]:
        with pytest.raises(error):
            call(**kw)


@pytest.mark.parametrize("tokens,rows,cols", [(1, 20011, 96), (17, 9434, 64), (70, 12001, 320), (500, 50257, 160)])
@pytest.mark.parametrize("bits,bucket", [(4, 1024), (8, 96)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gradient_over_many_rows(tokens, rows, cols, bits, bucket, dtype):
    """Few tiles, whose depth many workgroups share."""
    g = gen("deep", tokens, rows, cols, bits)
    weights = dev(coded(rows, cols, bucket, bits, g))
    x = torch.randn(tokens, rows, generator=g).to(dtype)
    want, tol = expect("grad", x.to(DEV), weights, rows, cols, bucket, bits)
    assert torch.all((run("grad", padded(x), weights, rows, cols, bucket, bits).double() - want).abs() <= tol)
