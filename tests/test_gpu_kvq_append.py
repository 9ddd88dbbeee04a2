"""The rotating append on the GPU: turned queries and coded rows bit for bit as the formulas in 64 bits give
them, and a decoding step that stays in codes from one projection to the next."""
import math

import pytest
import torch

import kvq_ref
import qsdp_linear_ref as ref
from error_compensated_bit_amd import onebit as ob
from test_gpu_kvq import BF16, DEV, F16, F32, dev, expect_written, gen, random_pools, same_bits

pytestmark = pytest.mark.gpu


def table(far, rot, base=10000.0):
    """[far, rot] cosines and sines, fp32."""
    half = rot // 2
    freq = base ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(far, dtype=torch.float64).unsqueeze(1) * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def turn(x, positions, rotary, interleaved):
    """Rows x [tokens, heads, dim] turned, in fp32: products of two fp32 numbers are exact in fp64."""
    rot = rotary.shape[1]
    known = (positions >= 0) & (positions < rotary.shape[0])
    t = rotary.double()[torch.where(known, positions, 0)]
    t = torch.where(known.unsqueeze(1), t, torch.full_like(t, math.nan)).unsqueeze(1)
    c, s = t[..., :rot // 2], t[..., rot // 2:]
    y = x.double().clone()
    if interleaved:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y.float()


def check(q, k, v, positions, rotary, slots, pools, bits, interleaved, in_place=False):
    turned = turn(k, positions, rotary, interleaved)
    want = expect_written(pools, turned, v, slots, bits)
    got = dev(pools)
    put = dev((positions, rotary, slots))
    # queries, keys and values side by side, as a fused projection leaves them
    qkv = torch.cat([t for t in (q, k, v) if t is not None], 1).to(DEV)
    hq, h = 0 if q is None else q.shape[1], k.shape[1]
    qd = None if q is None else qkv[:, :hq]
    out = None if q is None else qd if in_place else torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    ob.kvq_append(qd, qkv[:, hq:hq + h], qkv[:, hq + h:], put[0], put[1], put[2], *got, out, bits=bits,
                  interleaved=interleaved)
    for name, a, b in zip(("k_codes", "k_scales", "v_codes", "v_scales"), got, want):
        assert same_bits(a.cpu(), b), name
    if q is not None:
        assert same_bits(out.cpu(), turn(q, positions, rotary, interleaved).to(q.dtype)), "q_out"
    assert same_bits(qkv[:, hq:].cpu(), torch.cat((k, v), 1))


def rows(tokens, heads, dim, dtype, g):
    x = torch.randn(tokens, heads, dim, generator=g)
    return (x * torch.exp2(torch.randint(-12, 13, (tokens, heads, 1), generator=g).float())).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (64, 48), (128, 128), (128, 16), (128, 112), (256, 256), (256, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
def test_appended_rows_bit_for_bit(dtype, dim, rot, interleaved, bits):
    for tokens, hq, heads, page in ((1, 1, 1, 16), (2, 8, 2, 16), (37, 3, 3, 64), (300, 6, 1, 1024), (131, 0, 5, 32)):
        g = gen("append", dim, rot, tokens)
        n_pages = -(-tokens // page) + 2
        pools = random_pools(n_pages, heads, page, dim, bits, g)
        slots = torch.randperm(n_pages * page, generator=g)[:tokens]
        positions = torch.randint(0, 1000, (tokens,), generator=g)
        if tokens > 10:     # padding, slots behind the cache, positions outside the table
            slots[3], slots[5], slots[7], slots[-1] = -1, n_pages * page, 2 ** 62, -2 ** 63
            positions[2], positions[3], positions[6], positions[8], positions[-2] = 999, 1000, -1, 2 ** 62, -2 ** 63
        q = rows(tokens, hq, dim, dtype, g) if hq else None
        k, v = rows(tokens, heads, dim, dtype, g), rows(tokens, heads, dim, dtype, g)
        check(q, k, v, positions, table(1000, rot), slots, pools, bits, interleaved, in_place=tokens == 37)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_special_values(dtype, interleaved):
    """Infinities, NaN, the type's largest values, zeros of both signs, subnormals: a bad value stays in its
    own pair of a query and in its own row of the cache."""
    g = gen("special", interleaved)
    fi = torch.finfo(dtype)
    k = rows(12, 2, 64, dtype, g)
    k[1, 0, 5], k[2, 1, 60], k[3, 0, 31] = math.inf, math.nan, -math.inf
    k[4], k[5], k[6] = 0.0, -0.0, fi.tiny
    k[7], k[8] = fi.max, fi.smallest_normal / 4
    k[9, :, ::2] = 0.0
    pools = random_pools(3, 2, 16, 64, 8, g)
    slots, positions = torch.arange(12) + 7, torch.arange(12)
    rotary = table(12, 32)
    check(k.clone(), k, k.flip(0), positions, rotary, slots, pools, 8, interleaved)


def test_far_positions_and_factors_of_the_table():
    """A long table (rows behind 2^31 bytes) with a factor on its entries."""
    g = gen("far")
    far, rot = 5 * 2 ** 20, 128
    rotary = torch.zeros(far, rot, device=DEV)
    at = torch.tensor([0, 1, 2 ** 22, far - 2, far - 1])
    t = table(5, rot) * 1.125
    rotary[at.to(DEV)] = t.to(DEV)
    q, k, v = (rows(5, 2, 128, BF16, g) for _ in range(3))
    pools = dev(random_pools(2, 2, 16, 128, 4, g))
    out = torch.zeros(5, 2, 128, dtype=BF16, device=DEV)
    ob.kvq_append(*dev((q, k, v, at)), rotary, torch.arange(5, device=DEV), *pools, out, bits=4)
    assert torch.equal(out.cpu(), turn(q, torch.arange(5), t, False).to(BF16))


def test_an_empty_cache_still_turns_queries():
    g = gen("empty")
    q, k = rows(9, 4, 64, F16, g), rows(9, 2, 64, F16, g)
    check(q, k, k, torch.arange(9), table(9, 64), torch.arange(9), random_pools(0, 2, 16, 64, 8, g), 8, False)


def test_it_is_the_quantizer_where_nothing_turns():
    """Positions of angle 0: kvq_append writes what kvq_quantize writes."""
    g = gen("same")
    k, v = rows(70, 3, 128, BF16, g).to(DEV), rows(70, 3, 128, BF16, g).to(DEV)
    slots = torch.randperm(80, generator=g)[:70].to(DEV)
    pools = random_pools(5, 3, 16, 128, 4, g)
    one, two = dev(pools), dev(pools)
    ob.kvq_quantize(k, v, slots, *one, bits=4)
    ob.kvq_append(None, k, v, torch.zeros(70, dtype=torch.int64, device=DEV), table(1, 128).to(DEV), slots, *two, None,
                  bits=4)
    for a, b in zip(one, two):
        assert torch.equal(a, b)


def test_bindings_refusals():
    g = gen("refusals")
    q, k = rows(5, 4, 64, BF16, g).to(DEV), rows(5, 2, 64, BF16, g).to(DEV)
    pos, rotary, slots = torch.arange(5, device=DEV), table(8, 64).to(DEV), torch.arange(5, device=DEV)
    pools = dev(random_pools(1, 2, 16, 64, 8, g))

    def call(q=q, k=k, v=k, pos=pos, rotary=rotary, slots=slots, pools=pools, out=q, bits=8):
        ob.kvq_append(q, k, v, pos, rotary, slots, *pools, out, bits=bits)

    call()
    for error, kw in [(ValueError, dict(q=None)), (ValueError, dict(out=None)), (ValueError, dict(out=q.half())),
                      (ValueError, dict(v=k.half())), (ValueError, dict(v=k[:4])), (ValueError, dict(q=q[:4], out=q[:4])),
                      (ValueError, dict(out=q[:, :3])), (ValueError, dict(pos=pos[:4])), (TypeError, dict(pos=pos.int())),
                      (ValueError, dict(pos=torch.arange(10, device=DEV)[::2])), (TypeError, dict(rotary=rotary.half())),
                      (ValueError, dict(rotary=rotary[:, :32])), (ValueError, dict(rotary=rotary[0])),
                      (ob.OnebitError, dict(rotary=rotary[:0])), (ob.OnebitError, dict(rotary=table(8, 8).to(DEV))),
                      (ob.OnebitError, dict(rotary=table(8, 80).to(DEV))), (ValueError, dict(slots=slots[1:])),
                      (TypeError, dict(slots=slots.int())), (ValueError, dict(bits=5)), (ValueError, dict(bits=4)),
                      (TypeError, dict(pos=pos.cpu())), (TypeError, dict(q=q.cpu(), out=q.cpu()))]:
        with pytest.raises(error):
            call(**kw)


def test_captured_and_replayed_on_a_side_stream():
    g = gen("graph")
    q, k = rows(40, 4, 128, BF16, g).to(DEV), rows(40, 2, 128, BF16, g).to(DEV)
    pos, slots, rotary = torch.arange(40, device=DEV), torch.arange(40, device=DEV), table(400, 128).to(DEV)
    pools, eager = dev(random_pools(3, 2, 16, 128, 8, g)), dev(random_pools(3, 2, 16, 128, 8, gen("graph")))
    eager = [p.clone() for p in pools]
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ob.kvq_append(q, k, k, pos, rotary, slots, *pools, out, bits=8)
    for step in range(4):
        q.copy_(rows(40, 4, 128, BF16, g))
        k.copy_(rows(40, 2, 128, BF16, g))
        pos.add_(90)
        ob.kvq_append(q, k, k, pos, rotary, slots, *eager, want, bits=8)
        graph.replay()
        torch.cuda.synchronize()
        # (the last step's positions are behind the table)
        assert same_bits(out, want), step
        for a, b in zip(pools, eager):
            assert same_bits(a, b), step


@pytest.mark.parametrize("dtype,bits", [(BF16, 4), (F16, 8)])
def test_a_decoding_step_in_codes(dtype, bits):
    """Projection from coded weights, append, attention over the coded cache, projection back: a prompt in two
    chunks and then single tokens of three sequences, each stage against its formulas on the stage's own input."""
    hidden, hq, heads, dim, page, bucket = 288, 6, 2, 64, 16, 1024
    wide = (hq + 2 * heads) * dim
    g = gen("decode", bits)

    def matrix(rows, cols):
        from test_gpu_qsdp_linear import coded
        return coded(rows, cols, bucket, bits, g)

    w_in, w_out = matrix(wide, hidden), matrix(hidden, hq * dim)
    w_in_d, w_out_d = dev(w_in), dev(w_out)
    w_in64, w_out64 = (ref.weights(*w, r, c, bucket, bits) for w, r, c in ((w_in, wide, hidden), (w_out, hidden, hq * dim)))
    batch, room = 3, 8
    tables = torch.randperm(batch * room + 2, generator=g)[:batch * room].view(batch, room).int()
    pools = tuple(torch.zeros_like(p) for p in random_pools(batch * room + 2, heads, page, dim, bits, g))
    got = dev(pools)
    rotary = table(room * page, dim)
    lens = [0, 0, 0]
    ws = torch.zeros(max(ob.qsdp_linear_workspace_bytes(256, wide, hidden), ob.qsdp_linear_workspace_bytes(256, hidden, hq * dim)),
                     dtype=torch.uint8, device=DEV)
    aws = torch.zeros(ob.kvq_attention_workspace_bytes(batch, 256, hq, heads, dim), dtype=torch.uint8, device=DEV)
    for new in ((60, 1, 33), (30, 40, 2), (1, 1, 1), (1, 1, 1)):
        total = sum(new)
        positions = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, new)])
        seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(new))
        slots = tables[seq, positions // page].long() * page + positions % page
        lens = [n + m for n, m in zip(lens, new)]
        offsets = torch.tensor([0, new[0], new[0] + new[1], total], dtype=torch.int32)
        kv_lens = torch.tensor(lens, dtype=torch.int32)
        x = torch.randn(total, hidden, generator=g).to(dtype)

        qkv = torch.zeros(total, hq + 2 * heads, dim, dtype=dtype, device=DEV)
        ob.qsdp_linear(x.to(DEV), *w_in_d, qkv.view(total, wide), bucket=bucket, bits=bits, workspace=ws)
        want, tol = ref.product(x, w_in64[0].t().contiguous(), w_in64[1].t().contiguous(), bits, dtype, total <= ob.QSDP_LINEAR_EXACT_TOKENS)
        assert torch.all((qkv.view(total, wide).cpu().double() - want).abs() <= tol)

        rows_in = qkv.cpu()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
        ob.kvq_append(q, k, v, positions.to(DEV), rotary.to(DEV), slots.to(DEV), *got, q, bits=bits)
        pools = expect_written(pools, turn(rows_in[:, hq:hq + heads], positions, rotary, False), rows_in[:, hq + heads:], slots, bits)
        for a, b in zip(got, pools):
            assert same_bits(a.cpu(), b)
        turned = turn(rows_in[:, :hq], positions, rotary, False).to(dtype)
        assert same_bits(q.cpu(), turned)

        out = torch.zeros(total, hq, dim, dtype=dtype, device=DEV)
        uniform = min(new) == max(new)
        ob.kvq_attention(q, *got, tables.to(DEV), kv_lens.to(DEV), out, bits=bits, workspace=aws,
                         q_offsets=None if uniform else offsets.to(DEV))
        want, _, tol, _, _ = kvq_ref.attention(turned, pools, tables, kv_lens, bits=bits, scale=dim ** -0.5, q_offsets=offsets)
        half = kvq_ref.HALF_STEP[dtype]
        assert torch.all((out.cpu().double() - want).abs() <= tol + half * (want.abs() + tol) + 2.0 ** -25)

        y = torch.zeros(total, hidden, dtype=dtype, device=DEV)
        ob.qsdp_linear(out.view(total, hq * dim), *w_out_d, y, bucket=bucket, bits=bits, workspace=ws)
        want, tol = ref.product(out.cpu().view(total, hq * dim), w_out64[0].t().contiguous(), w_out64[1].t().contiguous(), bits, dtype,
                                total <= ob.QSDP_LINEAR_EXACT_TOKENS)
        assert torch.all((y.cpu().double() - want).abs() <= tol)
