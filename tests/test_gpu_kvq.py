"""The coded key/value cache on the GPU: rows written bit for bit as the 64-bit
reference codes them, read back as their values, and attended to within tolerances
that count roundings (kvq_ref.attention)."""
import math
import zlib

import numpy as np
import pytest
import torch

import kvq_ref
from error_compensated_bit_amd import onebit as ob

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def empty_pools(n_pages, heads, page, dim, bits, fill=0):
    """Codes and scales of keys and values on the CPU."""
    def codes():
        return torch.full((n_pages, heads, page, dim * bits // 8), fill, dtype=torch.uint8)
    return codes(), torch.zeros(n_pages, heads, page), codes(), torch.zeros(n_pages, heads, page)


def random_pools(n_pages, heads, page, dim, bits, g, spread=True):
    pools = []
    for _ in range(2):
        x = torch.randn(n_pages, heads, page, dim, generator=g)
        if spread:      # rows of very different size
            x *= torch.exp2(torch.randint(-6, 7, (n_pages, heads, page, 1), generator=g).float() / 4)
        code, scale = kvq_ref.code_rows(x.to(BF16), bits)
        pools += [kvq_ref.pack(code, bits), scale]
    return tuple(pools)


def dev(ts):
    return tuple(None if t is None else t.to(DEV) for t in ts)


# ------------------------------------------------------------------ write

def expect_written(pools, k, v, slots, bits):
    n_pages, heads, page, _ = pools[0].shape
    out = [p.clone() for p in pools]
    for which, x in ((0, k), (2, v)):
        code, scale = kvq_ref.code_rows(x, bits)
        code = kvq_ref.pack(code, bits)
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < n_pages * page:
                out[which][s // page, :, s % page] = code[i]
                out[which + 1][s // page, :, s % page] = scale[i]
    return out


def same_bits(a, b):
    """Equal, NaN where the other is NaN."""
    return torch.equal(a, b) if a.dtype == torch.uint8 else \
        torch.equal(torch.nan_to_num(a, nan=-1.0), torch.nan_to_num(b, nan=-1.0)) and \
        torch.equal(torch.isnan(a), torch.isnan(b))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 2, 64), (256, 1, 32), (128, 5, 1024)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens", [1, 2, 37, 300])
def test_write_codes_rows_bit_for_bit(dtype, dim, heads, page, bits, tokens):
    g = gen("write", dim, bits, tokens)
    n_pages = -(-tokens // page) + 2
    pools = random_pools(n_pages, heads, page, dim, bits, g)
    kv = (torch.randn(tokens, 2 * heads + 1, dim, generator=g) *
          torch.exp2(torch.randint(-12, 13, (tokens, 2 * heads + 1, 1), generator=g).float())).to(dtype)
    slots = torch.randperm(n_pages * page, generator=g)[:tokens]
    if tokens > 10:     # padding, and slots behind the cache
        slots[3], slots[5], slots[7], slots[-1] = -1, n_pages * page, 2 ** 62, -2 ** 63
    k, v = kv[:, :heads], kv[:, heads:2 * heads]                # strided, as a fused projection leaves them
    want = expect_written(pools, k, v, slots, bits)
    got = dev(pools)
    kvd = kv.to(DEV)
    ob.kvq_quantize(kvd[:, :heads], kvd[:, heads:2 * heads], slots.to(DEV), *got, bits=bits)
    for name, a, b in zip(("k_codes", "k_scales", "v_codes", "v_scales"), got, want):
        assert same_bits(a.cpu(), b), name


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_write_of_special_rows(bits, dtype):
    """Ties, zeros of both signs, rows at and below the smallest kept magnitude, the type's largest
    values, infinities and NaN."""
    top = kvq_ref.LEVELS[bits][0]
    fi = torch.finfo(dtype)
    x = torch.zeros(12, 1, 64)
    x[0, 0] = (torch.arange(64) % (2 * int(top)) - top) + 0.5             # ties: the reciprocal is 1
    x[0, 0, 7], x[0, 0, 8] = top, -top
    x[1, 0, 3] = -0.0
    x[2] = fi.max
    x[3, 0, ::2], x[3, 0, 1::2] = fi.max, -fi.max
    x[4, 0, 5] = math.inf
    x[5, 0, 5] = -math.inf
    x[6, 0, 63] = math.nan
    x[7, 0, 0], x[7, 0, 1] = math.nan, math.inf
    x[8, 0, :4] = torch.tensor([2.0 ** -110, 2.0 ** -111, -2.0 ** -112, 2.0 ** -126])
    x[9, 0, :3] = torch.tensor([2.0 ** -111, -2.0 ** -120, 1e-40])
    x[10, 0, 9] = fi.tiny
    x[11, 0, ::3] = 1e-44
    x = x.to(dtype)
    pools = empty_pools(1, 1, 16, 64, bits, fill=0x55)
    slots = torch.arange(12)
    want = expect_written(pools, x, x.flip(0), slots, bits)
    got = dev(pools)
    ob.kvq_quantize(x.to(DEV), x.flip(0).to(DEV), slots.to(DEV), *got, bits=bits)
    for a, b in zip(got, want):
        assert same_bits(a.cpu(), b)
    # and they read back: NaN rows throughout, zero rows as 0
    ks, vs = torch.empty(12, 1, 64, device=DEV), torch.empty(12, 1, 64, device=DEV)
    ob.kvq_dequantize(*got, slots.to(DEV), ks, vs, bits=bits)
    ks = ks.cpu()
    assert torch.isnan(ks[4:8]).all() and torch.isnan(vs.cpu()[4:8]).all()
    assert (ks[1] == 0).all() and torch.isfinite(ks[:4]).all()


# ------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 2, 64), (256, 1, 32)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens", [1, 2, 37, 300])
def test_read_gives_the_values(dtype, dim, heads, page, bits, tokens):
    g = gen("read", dim, bits, tokens)
    pools = random_pools(7, heads, page, dim, bits, g)
    slots = torch.randint(0, 7 * page, (tokens,), generator=g)          # repeats among them
    if tokens > 10:
        slots[2], slots[4], slots[-1] = -5, 7 * page, 2 ** 40
    skip = (slots < 0) | (slots >= 7 * page)
    ko, vo = (torch.full((tokens, heads, dim), 3.0, dtype=dtype, device=DEV) for _ in range(2))
    ob.kvq_dequantize(*dev(pools), slots.to(DEV), ko, vo, bits=bits)
    at = slots.masked_fill(skip, 0)
    for which, got in ((0, ko), (2, vo)):
        # (code - z) * scale is exact in fp64, so this is the one fp32 rounding of the definition
        y = kvq_ref.values(pools[which][at // page, :, at % page], pools[which + 1][at // page, :, at % page], bits)
        y = y.float().to(dtype)
        y[skip] = 3.0
        assert torch.equal(got.cpu(), y)


def test_read_to_fp16_overflows_to_infinity():
    pools = empty_pools(1, 1, 16, 64, 8, fill=255)
    pools[1][:], pools[3][:] = 1e4, 500.0
    ko, vo = torch.zeros(2, 1, 64, dtype=F16, device=DEV), torch.zeros(2, 1, 64, dtype=F16, device=DEV)
    ob.kvq_dequantize(*dev(pools), torch.tensor([0, 15], device=DEV), ko, vo, bits=8)
    assert torch.isinf(ko).all() and (vo == 63488.0).all()              # 127 * 500 = 63500, to fp16's step of 32


# -------------------------------------------------------------- attention

def attend(q, pools, table, kv_lens, bits, *, scale=None, q_offsets=None, softcap=0.0, window=0, lse=True, fill=7.0,
           qd=None):
    """The call on the GPU: (out, lse) on the CPU, both pre-filled with `fill`."""
    total, hq, dim = q.shape
    out = torch.full((total, hq, dim), fill, dtype=q.dtype, device=DEV)
    l = torch.full((total, hq), fill, device=DEV) if lse else None
    size = ob.kvq_attention_workspace_bytes(len(kv_lens), total, hq, pools[0].shape[1], dim)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    pd = dev(pools)
    ob.kvq_attention(q.to(DEV) if qd is None else qd, *pd, table.to(DEV), kv_lens.to(DEV), out, bits=bits, scale=scale,
                     q_offsets=None if q_offsets is None else q_offsets.to(DEV), softcap=softcap, window=window, lse=l,
                     workspace=ws)
    return out.cpu(), None if l is None else l.cpu()


def check(got, got_lse, ref, dtype, fill=7.0):
    out, lse, tol, lse_tol, owned = ref
    half = kvq_ref.HALF_STEP[dtype]
    got = got.double()
    assert (got[~owned] == fill).all(), "rows of no sequence"
    out, tol, got = out[owned], tol[owned], got[owned]
    bad = torch.isnan(out)
    assert torch.equal(bad, torch.isnan(got))
    out, tol, got = out[~bad], tol[~bad], got[~bad]
    # the rounding of the output itself, and half the type's smallest step
    limit = tol + half * (out.abs() + tol) + (2.0 ** -25 if dtype == F16 else 2.0 ** -134)
    off = (got - out).abs()
    assert (off <= limit).all(), f"off by {float((off / limit.clamp_min(1e-300)).max()):.2f} of the tolerance"
    if got_lse is not None:
        assert (got_lse[~owned] == fill).all()
        want, have = lse[owned], got_lse[owned].double()
        gone = torch.isinf(want)
        assert torch.equal(gone, have == -math.inf)
        ok = ~(gone | torch.isnan(want))
        assert ((want - have).abs()[ok] <= lse_tol[owned][ok]).all()


def make(g, qs, ks, hq, heads, dim, page, bits, dtype, spread=True, peaked=2.0):
    """(q with room behind the last sequence, pools, table, kv_lens, q_offsets)."""
    need = [-(-k // page) for k in ks]
    n_pages = sum(need) + 2
    pools = random_pools(n_pages, heads, page, dim, bits, g, spread)
    order = torch.randperm(n_pages, generator=g)
    table = torch.full((len(qs), max(need + [1])), -1, dtype=torch.int32)
    used = 0
    for b, m in enumerate(need):
        table[b, :m] = order[used:used + m].int()
        used += m
    offs = torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32)
    q = (torch.randn(int(offs[-1]), hq, dim, generator=g) * peaked).to(dtype)
    return q, pools, table, torch.tensor(ks, dtype=torch.int32), offs


LAYOUTS = [(1, 1, 64), (4, 4, 128), (8, 1, 128), (6, 2, 256), (16, 2, 64), (12, 4, 128), (34, 2, 64), (40, 1, 128)]


@pytest.mark.parametrize("hq,heads,dim", LAYOUTS)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_single_tokens(hq, heads, dim, bits, dtype):
    ks = [1, 2, 15, 16, 17, 31, 33, 64, 127, 129, 300, 1111]
    g = gen("single", hq, dim, bits)
    q, pools, table, lens, _ = make(g, [1] * len(ks), ks, hq, heads, dim, 16, bits, dtype)
    sc = dim ** -0.5
    got, lse = attend(q, pools, table, lens, bits)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=bits, scale=sc), dtype)


@pytest.mark.parametrize("hq,heads,dim", LAYOUTS)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_chunks_of_every_length(hq, heads, dim, bits, dtype):
    qs = [1, 3, 17, 0, 33, 64, 130, 1, 257]
    ks = [1, 40, 17, 50, 333, 64, 700, 999, 300]
    g = gen("chunks", hq, dim, bits)
    q, pools, table, lens, offs = make(g, qs, ks, hq, heads, dim, 32, bits, dtype)
    got, lse = attend(q, pools, table, lens, bits, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=bits, scale=dim ** -0.5, q_offsets=offs), dtype)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 100, 5000])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("bits,dim,page", [(8, 128, 16), (4, 64, 256), (8, 256, 64)])
def test_windows_and_caps(window, softcap, bits, dim, page):
    qs, ks = [1, 5, 200, 70, 1], [700, 300, 900, 70, 2500]
    g = gen("window", window, bits, dim)
    q, pools, table, lens, offs = make(g, qs, ks, 4, 2, dim, page, bits, BF16)
    got, lse = attend(q, pools, table, lens, bits, q_offsets=offs, softcap=softcap, window=window)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=bits, scale=dim ** -0.5, q_offsets=offs,
                                      softcap=softcap, window=window), BF16)


@pytest.mark.parametrize("softcap", [2.0 ** -64, 64.0, 65.0, 100.0, 5e4, 1e9, 2.0 ** 64])
@pytest.mark.parametrize("bits,dtype", [(8, F16), (4, BF16), (8, BF16)])
def test_caps_far_from_the_scores(softcap, bits, dtype):
    """A cap far above the scores leaves them as they are (the difference that tanh's formula ends in
    does not), one far below makes them all alike; scores from 0 to beyond an eighth of the cap."""
    qs, ks = [1, 5, 200, 33, 1], [700, 300, 400, 70, 2500]
    g = gen("caps", softcap, bits, dtype)
    q, pools, table, lens, offs = make(g, qs, ks, 4, 2, 128, 32, bits, dtype)
    q[7:40] = 0
    got, lse = attend(q, pools, table, lens, bits, q_offsets=offs, softcap=softcap, scale=0.5)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=bits, scale=0.5, q_offsets=offs, softcap=softcap), dtype)


@pytest.mark.parametrize("q_len", [1, 2, 5, 9, 48])
@pytest.mark.parametrize("bits", [4, 8])
def test_rows_that_attend_to_nothing(q_len, bits):
    """More new tokens than the cache holds, empty and negative lengths: out 0, lse -inf."""
    lens = torch.tensor([0, 1, -7, 4, 47, q_len, -2 ** 31, 200], dtype=torch.int32)
    g = gen("nothing", q_len, bits)
    q, pools, table, _, _ = make(g, [q_len] * 8, [0, 1, 0, 4, 47, q_len, 0, 200], 8, 2, 128, 16, bits, F16)
    got, lse = attend(q, pools, table, lens, bits)
    ref = kvq_ref.attention(q, pools, table, lens, bits=bits, scale=128 ** -0.5)
    check(got, lse, ref, F16)
    assert (got[:q_len] == 0).all() and (lse[:q_len] == -math.inf).all()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 20, 2 ** 30])
@pytest.mark.parametrize("q_len", [7, 48])
def test_the_widest_windows(window, q_len):
    """A window that reaches far in front of the first token, with queries that stand there."""
    lens = torch.tensor([0, 4, 47, q_len, 200], dtype=torch.int32)
    g = gen("widest", q_len)
    q, pools, table, _, _ = make(g, [q_len] * 5, [0, 4, 47, q_len, 200], 8, 2, 64, 16, 8, BF16)
    got, lse = attend(q, pools, table, lens, 8, window=window)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125), BF16)


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("bits", [4, 8])
def test_unattended_positions_have_no_influence(q_len, bits):
    """Codes of all bits set and scales of NaN, infinity and the type's extremes behind the last token,
    in front of the window and in pages of other sequences: the result keeps its bits."""
    g = gen("stale", q_len, bits)
    q, pools, table, lens, offs = make(g, [q_len] * 3, [75, 333, 500], 4, 2, 128, 64, bits, BF16)
    ref = attend(q, pools, table, lens, bits, q_offsets=offs, window=40)
    attended = torch.zeros(pools[1].shape[0], 64, dtype=torch.bool)
    for b in range(3):
        for j in range(max(0, int(lens[b]) - q_len - 40 + 1), int(lens[b])):
            attended[int(table[b, j // 64]), j % 64] = True
    dirty = [p.clone() for p in pools]
    junk = torch.tensor([math.nan, math.inf, -math.inf, 3e38, -3e38, -1.0])
    gone = ~attended.unsqueeze(1).expand(-1, 2, -1)
    for which in (0, 2):
        dirty[which][gone] = 255
        dirty[which + 1][gone] = junk[torch.randint(0, 6, (int(gone.sum()),), generator=g)]
    got = attend(q, tuple(dirty), table, lens, bits, q_offsets=offs, window=40)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    check(got[0], got[1], kvq_ref.attention(q, tuple(dirty), table, lens, bits=bits, scale=128 ** -0.5, q_offsets=offs,
                                            window=40), BF16)


@pytest.mark.parametrize("q_len", [1, 40])
def test_pages_outside_the_cache_are_left_out(q_len):
    g = gen("pages", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 4, [200, 64, 333, 100], 4, 2, 128, 16, 8, BF16)
    table[0, 3], table[0, 7], table[1, 0], table[2, 20] = -1, pools[0].shape[0], 2 ** 31 - 1, -2 ** 31
    table[3, :] = -1                                                     # nothing left to attend to
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=128 ** -0.5, q_offsets=offs), BF16)
    assert (got[3 * q_len:] == 0).all()


@pytest.mark.parametrize("q_len", [1, 40])
def test_lengths_beyond_the_table_and_offsets_beyond_the_rows(q_len):
    g = gen("beyond", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 3, [48, 48, 48], 4, 2, 64, 16, 8, F16)
    lens = torch.tensor([2 ** 31 - 1, 49, 48], dtype=torch.int32)        # the table has 48 positions
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125, q_offsets=offs), F16)
    # offsets are clamped to the rows: the last sequence's missing rows do not exist
    wild = torch.tensor([-5, q_len, 2 * q_len, 2 ** 31 - 1], dtype=torch.int32)
    again, _ = attend(q, pools, table, lens, 8, q_offsets=wild)
    assert torch.equal(got, again)


@pytest.mark.parametrize("q_len", [1, 40])
def test_rows_of_no_sequence_keep_their_contents(q_len):
    g = gen("behind", q_len)
    q, pools, table, lens, offs = make(g, [q_len, 0, q_len], [50, 60, 70], 8, 2, 128, 16, 8, BF16)
    q = torch.cat([q, torch.full((13, 8, 128), math.nan, dtype=BF16)])
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    assert (got[2 * q_len:] == 7).all() and (lse[2 * q_len:] == 7).all()
    ref = kvq_ref.attention(q, pools, table, lens, bits=8, scale=128 ** -0.5, q_offsets=offs)
    check(got, lse, ref, BF16)
    # ... and rows in front of the first
    got, _ = attend(q, pools, table[:1], lens[:1], 8, q_offsets=torch.tensor([q_len, 2 * q_len], dtype=torch.int32))
    assert (got[:q_len] == 7).all() and (got[2 * q_len:] == 7).all() and (got[q_len:2 * q_len] != 7).any()


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("which", [1, 3])
def test_a_nan_scale_that_is_attended_to_gives_nan(q_len, which):
    g = gen("nan", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 2, [200, 300], 4, 2, 64, 16, 8, BF16)
    pools[which][int(table[1, 5]), 1, 3] = math.nan
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    assert torch.isfinite(got[:q_len]).all() and torch.isfinite(got[q_len:, :2]).all()
    assert torch.isnan(got[q_len:, 2:]).all()
    if which == 1:
        assert torch.isnan(lse[q_len:, 2:]).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_len,kv,at", [(5, 90, 87), (70, 100, 83), (300, 300, 140)])
@pytest.mark.parametrize("which,bad", [(1, math.nan), (3, math.nan), (3, math.inf)])
def test_a_bad_scale_concerns_only_those_who_attend_to_it(dtype, q_len, kv, at, which, bad):
    """A row whose scale is not finite, in the middle of the new tokens: nothing finite from it on (an
    infinite value times a weight is one, by the formula), and as before it without it."""
    g = gen("bad", q_len)
    q, pools, table, lens, offs = make(g, [q_len], [kv], 4, 2, 64, 16, 8, dtype)
    ref = kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125)
    dirty = [p.clone() for p in pools]
    dirty[which][int(table[0, at // 16]), :, at % 16] = bad
    got, _ = attend(q, tuple(dirty), table, lens, 8)
    first = at - (kv - q_len)                       # the query that stands at the row
    assert torch.isnan(got[first:]).all() if math.isnan(bad) else not torch.isfinite(got[first:]).any()
    cut = tuple(t[:first] for t in ref)
    check(got[:first], None, cut, dtype)


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("v_size", [1e-30, 1e-3, 1.0, 1e5, 1e30])
def test_values_of_any_size(q_len, v_size):
    """Scales over many powers of two, and rows of zeros: the weights' fp16 range is relative to the
    largest scale of the row's own keys, whatever the type's range."""
    g = gen("size", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 3, [200, 333, 80], 4, 2, 128, 16, 8, BF16)
    pools[3].mul_(v_size)
    pools[3][:, :, 3] = 0.0
    pools[1][:, 0, 5] = 0.0
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=128 ** -0.5, q_offsets=offs), BF16)


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("bits", [4, 8])
def test_value_scales_that_grow_along_the_sequence(q_len, bits):
    """Every page's values are larger than the last one's, then much smaller."""
    g = gen("grow", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 2, [600, 300], 4, 2, 64, 16, bits, F16)
    for b in range(2):
        for i in range(int(lens[b]) // 16 + 1):
            if i < table.shape[1] and table[b, i] >= 0:
                pools[3][int(table[b, i])] *= 2.0 ** (i if i < 20 else -10) * 2.0 ** -12
    got, lse = attend(q, pools, table, lens, bits, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=bits, scale=0.125, q_offsets=offs), F16)


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("size", [0.0, 1e-20, 1e20])
def test_queries_of_any_size(q_len, size):
    """bf16 queries far outside fp16's range: a scale brings the scores back."""
    g = gen("qsize", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 2, [200, 300], 4, 2, 128, 16, 8, BF16)
    q = (q.float() * size).to(BF16)
    # within a row, from the largest down to nothing
    q[:, :, ::3] *= 2.0 ** -20
    sc = 128 ** -0.5 / (size or 1.0)
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs, scale=sc)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=sc, q_offsets=offs), BF16)


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("sc", [0.0, -0.2, 40.0])
def test_scales_of_the_scores(q_len, sc):
    """No scale, a negative one, and one that leaves a single key."""
    g = gen("scale", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 2, [200, 300], 4, 2, 64, 16, 8, BF16)
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs, scale=sc)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=sc, q_offsets=offs), BF16)


@pytest.mark.parametrize("q_len", [1, 50])
def test_scores_that_grow_along_the_sequence(q_len):
    """Each key scores higher than those before it: the running maximum moves in every tile."""
    g = gen("ramp", q_len)
    q, pools, table, lens, offs = make(g, [q_len] * 2, [900, 300], 4, 2, 64, 16, 8, BF16, peaked=0.2)
    q[:, :, 0] = 4.0
    for b in range(2):
        for j in range(int(lens[b])):
            page = int(table[b, j // 16])
            pools[0][page, :, j % 16, 0] = 255
            pools[1][page, :, j % 16] = 0.0002 * j
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125, q_offsets=offs), BF16)


@pytest.mark.parametrize("layout", ["heads_first", "fused", "one_row"])
@pytest.mark.parametrize("q_len", [1, 37])
def test_strided_queries(layout, q_len):
    g = gen("stride", q_len)
    b = 1 if layout == "one_row" else 3
    q, pools, table, lens, offs = make(g, [q_len] * b, [100, 250, 70][:b], 8, 2, 64, 16, 8, F16)
    if layout == "heads_first":
        qd = q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    else:
        wide = torch.full((q.shape[0], 13, 64), math.nan, dtype=F16)
        wide[:, 3:11] = q
        qd = wide.to(DEV)[:, 3:11]
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs, qd=qd)
    plain, _ = attend(q, pools, table, lens, 8, q_offsets=offs)
    assert torch.equal(got, plain)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125, q_offsets=offs), F16)


def test_a_slice_of_a_wider_block_table():
    g = gen("table")
    q, pools, table, lens, _ = make(g, [1] * 3, [100, 250, 70], 4, 2, 64, 16, 8, BF16)
    wide = torch.full((3, 40), 2 ** 30, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    out = torch.empty_like(q, device=DEV)
    ws = torch.zeros(ob.kvq_attention_workspace_bytes(3, 3, 4, 2, 64), dtype=torch.uint8, device=DEV)
    ob.kvq_attention(q.to(DEV), *dev(pools), wide.to(DEV)[:, :table.shape[1]], lens.to(DEV), out, bits=8, workspace=ws)
    plain, _ = attend(q, pools, table, lens, 8)
    assert torch.equal(out.cpu(), plain)


def test_shared_pages():
    """Sequences that share their first pages read the same rows."""
    g = gen("shared")
    q, pools, table, lens, offs = make(g, [1, 20, 1], [200, 200, 200], 4, 2, 128, 16, 8, BF16)
    table[1, :8], table[2, :8] = table[0, :8], table[0, :8]
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=128 ** -0.5, q_offsets=offs), BF16)


@pytest.mark.parametrize("bits,dim,hq,heads", [(8, 128, 8, 1), (4, 64, 2, 2)])
@pytest.mark.parametrize("q_len", [1, 6])
def test_a_long_cache_split_along_its_length(bits, dim, hq, heads, q_len):
    g = gen("long", dim)
    q, pools, table, lens, offs = make(g, [q_len] * 2, [30011, 9999], hq, heads, dim, 128, bits, BF16)
    got, lse = attend(q, pools, table, lens, bits, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=bits, scale=dim ** -0.5, q_offsets=offs), BF16)
    # the same bits every time: no sum depends on an order of arrival
    for _ in range(3):
        again, l2 = attend(q, pools, table, lens, bits, q_offsets=offs)
        assert torch.equal(got, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("hq,heads,dim,dtype", [(1, 1, 64, F16), (8, 2, 128, BF16), (2, 1, 256, BF16)])
def test_a_chunk_over_a_long_cache(hq, heads, dim, dtype):
    """One chunk, few heads: each row tile is split over many workgroups and joined."""
    g = gen("long chunk", dim)
    q, pools, table, lens, offs = make(g, [70], [20011], hq, heads, dim, 64, 8, dtype)
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=dim ** -0.5, q_offsets=offs), dtype)
    for _ in range(3):
        again, l2 = attend(q, pools, table, lens, 8, q_offsets=offs)
        assert torch.equal(got, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("hq,heads,dim", [(600, 2, 64), (257, 1, 128), (300, 1, 256)])
def test_more_query_heads_of_a_cache_head_than_a_tile_has_rows(hq, heads, dim):
    g = gen("group", hq)
    q, pools, table, lens, offs = make(g, [1, 3, 0, 2], [33, 70, 5, 2], hq, heads, dim, 16, 8, BF16)
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=dim ** -0.5, q_offsets=offs), BF16)


@pytest.mark.parametrize("hq,heads,dim", [(3, 3, 64), (2, 1, 128), (1, 1, 256)])
@pytest.mark.parametrize("rows", [16, 18, 32, 34, 48, 50, 64])
@pytest.mark.parametrize("pages", [40, 70000])
@pytest.mark.parametrize("ragged", [False, True])
def test_row_counts_at_the_kernels_boundaries(hq, heads, dim, rows, pages, ragged):
    """Also under a block table for far more tokens than there are."""
    m = rows * heads // hq
    g = gen("rows", hq, dim, rows, pages)
    q, pools, table, lens, offs = make(g, [m] * 3, [m, 700, 333], hq, heads, dim, 16, 8, BF16)
    wide = torch.full((3, max(pages, table.shape[1])), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    got, lse = attend(q, pools, wide, lens, 8, q_offsets=offs if ragged else None)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=dim ** -0.5), BF16)


@pytest.mark.parametrize("group", [17, 32, 33, 48, 49])
@pytest.mark.parametrize("pages", [40, 70000])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_groups_at_the_kernels_boundaries(group, pages, ragged, dtype):
    g = gen("groups", group, pages)
    q, pools, table, lens, offs = make(g, [1] * 5, [1, 2000, 40, 0, 333], 2 * group, 2, 128, 16, 4, dtype)
    wide = torch.full((5, max(pages, table.shape[1])), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    got, lse = attend(q, pools, wide, lens, 4, q_offsets=offs if ragged else None)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=4, scale=128 ** -0.5), dtype)


@pytest.mark.parametrize("n,q_len", [(1024, 1), (1025, 1), (2100, 2), (512, 40), (1300, 33)])
def test_more_sequences_than_a_launch_takes(n, q_len):
    g = gen("launches", n)
    ks = torch.randint(q_len, q_len + 30, (n,), generator=g).tolist()
    q, pools, table, lens, offs = make(g, [q_len] * n, ks, 1, 1, 64, 16, 8, BF16)
    got, lse = attend(q, pools, table, lens, 8)
    check(got, lse, kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125), BF16)
    again, _ = attend(q, pools, table, lens, 8, q_offsets=offs)
    assert torch.equal(got, again)


def test_one_workspace_for_calls_of_every_size():
    """A workspace is ready for the next call, whatever that one's sizes; two captured graphs that are
    replayed one after the other may share it."""
    g = gen("workspace")
    calls = []
    for qs, ks, hq, heads, dim, dtype in [([1] * 3, [3000, 200, 5000], 8, 2, 128, BF16), ([90], [4000], 2, 2, 64, F16),
                                          ([1, 40, 7], [2500, 700, 7], 4, 2, 256, BF16), ([1], [6000], 1, 1, 64, F16),
                                          ([3] * 5, [900, 20, 4000, 3, 1], 20, 1, 128, F16)]:
        q, pools, table, lens, offs = make(g, qs, ks, hq, heads, dim, 16, 8, dtype)
        want, _ = attend(q, pools, table, lens, 8, q_offsets=offs)
        size = ob.kvq_attention_workspace_bytes(len(qs), q.shape[0], hq, heads, dim)
        calls.append((dev((q, *pools, table, lens, offs)), want, size))
    ws = torch.zeros(max(c[2] for c in calls), dtype=torch.uint8, device=DEV)

    def run(c, out):
        q, kc, ks, vc, vs, table, lens, offs = c[0]
        ob.kvq_attention(q, kc, ks, vc, vs, table, lens, out, bits=8, q_offsets=offs, workspace=ws)

    outs = [torch.zeros_like(c[0][0]) for c in calls]
    for _ in range(3):
        for c, out in zip(calls, outs):
            out.zero_()
            run(c, out)
            assert torch.equal(out.cpu(), c[1])
    graphs = []
    for c, out in zip(calls, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(c, out)
        graphs.append(graph)
    for i in (0, 1, 2, 3, 4, 2, 0, 0, 3, 1, 4):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i].cpu(), calls[i][1]), i


def test_a_stream_given_by_number():
    g = gen("number")
    q, pools, table, lens, _ = make(g, [1] * 2, [300, 40], 4, 2, 64, 16, 8, BF16)
    want, _ = attend(q, pools, table, lens, 8)
    side = torch.cuda.Stream()
    qd, pd, td, ld = q.to(DEV), dev(pools), table.to(DEV), lens.to(DEV)
    out = torch.zeros_like(qd)
    ws = torch.zeros(ob.kvq_attention_workspace_bytes(2, 2, 4, 2, 64), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    ob.kvq_attention(qd, *pd, td, ld, out, bits=8, workspace=ws, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out.cpu(), want)
    # the current stream is the one taken otherwise
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        ob.kvq_attention(qd, *pd, td, ld, out, bits=8, workspace=ws)
    side.synchronize()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("q_max", [1, 90])
def test_many_sequences(q_max):
    g = gen("many", q_max)
    n = 300
    qs = [1] * n if q_max == 1 else torch.randint(0, q_max, (n,), generator=g).tolist()
    ks = [max(a, b) for a, b in zip(qs, torch.randint(0, 200, (n,), generator=g).tolist())]
    q, pools, table, lens, offs = make(g, qs, ks, 4, 2, 64, 16, 8, BF16)
    got, lse = attend(q, pools, table, lens, 8, q_offsets=offs)
    ref = kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125, q_offsets=offs)
    check(got, lse, ref, BF16)
    if q_max == 1:      # the same without offsets, bit for bit
        again, _ = attend(q, pools, table, lens, 8)
        assert torch.equal(got, again)


def test_empty_calls():
    pools = dev(random_pools(2, 2, 16, 64, 8, gen("empty")))
    ws = torch.zeros(ob.kvq_attention_workspace_bytes(2, 0, 4, 2, 64), dtype=torch.uint8, device=DEV)
    q = torch.empty(0, 4, 64, dtype=BF16, device=DEV)
    z = torch.zeros(2, dtype=torch.int32, device=DEV)
    ob.kvq_attention(q, *pools, torch.zeros(2, 1, dtype=torch.int32, device=DEV), z, q.clone(), bits=8, workspace=ws)
    none = torch.empty(0, 2, 64, dtype=BF16, device=DEV)
    at = torch.empty(0, dtype=torch.int64, device=DEV)
    ob.kvq_quantize(none, none.clone(), at, *pools, bits=8)
    ob.kvq_dequantize(*pools, at, none, none.clone(), bits=8)
    # a table without pages: nothing to attend to
    q = torch.ones(2, 4, 64, dtype=BF16, device=DEV)
    out = torch.ones_like(q)
    ws = torch.zeros(ob.kvq_attention_workspace_bytes(2, 2, 4, 2, 64), dtype=torch.uint8, device=DEV)
    ob.kvq_attention(q, *pools, torch.zeros(2, 0, dtype=torch.int32, device=DEV), z + 5, out, bits=8, workspace=ws)
    assert (out == 0).all()


@pytest.mark.parametrize("q_len", [1, 50])
def test_a_cache_without_pages(q_len):
    none = tuple(t.to(DEV) for t in empty_pools(0, 2, 16, 64, 8))
    q = torch.ones(2 * q_len, 4, 64, dtype=BF16, device=DEV)
    out, lse = torch.ones_like(q), torch.ones(2 * q_len, 4, device=DEV)
    ws = torch.zeros(ob.kvq_attention_workspace_bytes(2, 2 * q_len, 4, 2, 64), dtype=torch.uint8, device=DEV)
    table, lens = torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.full((2,), 40, dtype=torch.int32, device=DEV)
    ob.kvq_attention(q, *none, table, lens, out, bits=8, lse=lse, workspace=ws)
    assert (out == 0).all() and (lse == -math.inf).all()
    ob.kvq_quantize(q[:, :2], q[:, 2:], torch.arange(2 * q_len, device=DEV), *none, bits=8)   # no slot exists
    ob.kvq_dequantize(*none, torch.arange(2 * q_len, device=DEV), out[:, :2].contiguous(), out[:, 2:].contiguous(), bits=8)


def test_rows_past_4_gib():
    """Codes and scales at byte offsets beyond 32 bits, written, read and attended to."""
    page, heads, dim = 1024, 8, 256
    n_pages = 2 ** 33 // (page * heads * dim)                            # 8 GiB of codes each
    kc, vc = (torch.zeros(n_pages, heads, page, dim, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(n_pages, heads, page, device=DEV) for _ in range(2))
    g = gen("far")
    k, v = (torch.randn(300, heads, dim, generator=g).to(BF16) for _ in range(2))
    slots = torch.arange(n_pages * page - 300, n_pages * page)
    ob.kvq_quantize(k.to(DEV), v.to(DEV), slots.to(DEV), kc, ks, vc, vs, bits=8)
    assert int(kc[:n_pages // 2].amax()) == 0
    ko, vo = torch.zeros_like(k, device=DEV, dtype=F32), torch.zeros_like(k, device=DEV, dtype=F32)
    ob.kvq_dequantize(kc, ks, vc, vs, slots.to(DEV), ko, vo, bits=8)
    code, scale = kvq_ref.code_rows(k, 8)
    assert torch.equal(ko.cpu(), kvq_ref.values(code, scale, 8).float())
    small = tuple(t[-1:].cpu() for t in (kc, ks, vc, vs))
    for q_len in (1, 40):
        q = torch.randn(q_len, 8, dim, generator=g).to(BF16)
        table, lens = torch.tensor([[n_pages - 1]], dtype=torch.int32), torch.tensor([1024], dtype=torch.int32)
        out = torch.zeros_like(q, device=DEV)
        ws = torch.zeros(ob.kvq_attention_workspace_bytes(1, q_len, 8, heads, dim), dtype=torch.uint8, device=DEV)
        ob.kvq_attention(q.to(DEV), kc, ks, vc, vs, table.to(DEV), lens.to(DEV), out, bits=8, window=300, workspace=ws)
        plain, _ = attend(q, small, torch.zeros(1, 1, dtype=torch.int32), lens, 8, window=300)
        assert torch.equal(out.cpu(), plain)


# --------------------------------------------------------------- together

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_prompt_in_chunks_then_generation(bits, dtype):
    """As a server uses them: prompts enter in chunks (each written, then attended from), then tokens
    one by one; at every step the attention agrees with the reference over the cache as it stands, and
    what was written reads back."""
    heads, hq, dim, page, batch = 2, 6, 128, 16, 3
    g = gen("together", bits)
    pools = dev(empty_pools(40, heads, page, dim, bits))
    order = torch.randperm(40, generator=g).int()
    table = order[:36].view(3, 12)
    have = [0] * batch
    steps = [[50, 1, 0], [37, 60, 9], [1, 33, 20]] + [[1, 1, 1]] * 6
    for counts in steps:
        total = sum(counts)
        qkv = torch.randn(total, hq + 2 * heads, dim, generator=g).to(dtype)
        offs = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
        slots = []
        for b, c in enumerate(counts):
            for t in range(have[b], have[b] + c):
                slots.append(int(table[b, t // page]) * page + t % page)
            have[b] += c
        slots = torch.tensor(slots)
        lens = torch.tensor(have, dtype=torch.int32)
        d = qkv.to(DEV)
        q, k, v = d[:, :hq], d[:, hq:hq + heads], d[:, hq + heads:]
        ob.kvq_quantize(k, v, slots.to(DEV), *pools, bits=bits)
        out = torch.empty(total, hq, dim, dtype=dtype, device=DEV)
        ws = torch.zeros(ob.kvq_attention_workspace_bytes(batch, total, hq, heads, dim), dtype=torch.uint8, device=DEV)
        ob.kvq_attention(q, *pools, table.to(DEV), lens.to(DEV), out, bits=bits, q_offsets=offs.to(DEV), workspace=ws)
        ko, vo = (torch.empty(total, heads, dim, device=DEV) for _ in range(2))
        ob.kvq_dequantize(*pools, slots.to(DEV), ko, vo, bits=bits)
        host = tuple(p.cpu() for p in pools)
        ref = kvq_ref.attention(qkv[:, :hq], host, table, lens, bits=bits, scale=dim ** -0.5, q_offsets=offs)
        check(out.cpu(), None, ref, dtype)
        code, scale = kvq_ref.code_rows(qkv[:, hq:hq + heads], bits)
        assert torch.equal(ko.cpu(), kvq_ref.values(kvq_ref.pack(code, bits), scale, bits).float())


def test_a_captured_step_follows_its_inputs():
    """A whole step (write, attend, read) captured once and replayed while tokens, lengths and slots
    change in place, with eager work between the replays."""
    heads, hq, dim, page, bits, batch = 2, 8, 128, 16, 8, 4
    g = gen("graph")
    pools = dev(random_pools(30, heads, page, dim, bits, g))
    table = torch.randperm(30, generator=g)[:28].int().view(4, 7)
    qkv = torch.zeros(batch, hq + 2 * heads, dim, dtype=BF16, device=DEV)
    slots = torch.zeros(batch, dtype=torch.int64, device=DEV)
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    td = table.to(DEV)
    out = torch.zeros(batch, hq, dim, dtype=BF16, device=DEV)
    ko, vo = (torch.zeros(batch, heads, dim, device=DEV) for _ in range(2))
    ws = torch.zeros(ob.kvq_attention_workspace_bytes(batch, batch, hq, heads, dim), dtype=torch.uint8, device=DEV)

    def step():
        ob.kvq_quantize(qkv[:, hq:hq + heads], qkv[:, hq + heads:], slots, *pools, bits=bits)
        ob.kvq_attention(qkv[:, :hq], *pools, td, lens, out, bits=bits, workspace=ws)
        ob.kvq_dequantize(*pools, slots, ko, vo, bits=bits)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        slots.fill_(-1)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    have = [3, 40, 77, 100]
    for i in range(5):
        new = torch.randn(batch, hq + 2 * heads, dim, generator=g).to(BF16)
        at = torch.tensor([int(table[b, have[b] // page]) * page + have[b] % page for b in range(batch)])
        have = [h + 1 for h in have]
        qkv.copy_(new)
        slots.copy_(at)
        lens.copy_(torch.tensor(have, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        host = tuple(p.cpu() for p in pools)
        ref = kvq_ref.attention(new[:, :hq], host, table, lens.cpu(), bits=bits, scale=dim ** -0.5)
        check(out.cpu(), None, ref, BF16)
        code, scale = kvq_ref.code_rows(new[:, hq:hq + heads], bits)
        assert torch.equal(ko.cpu(), kvq_ref.values(code, scale, bits).float())
        replayed = out.clone()
        out.zero_()
        step()                                                           # eager, over the same cache
        assert torch.equal(out, replayed)


def test_two_calls_at_once_on_two_streams():
    """Calls with a workspace each may overlap."""
    g = gen("streams")
    q, pools, table, lens, offs = make(g, [1] * 4 + [60], [3000, 100, 2000, 50, 900], 8, 2, 128, 16, 8, BF16)
    want, _ = attend(q, pools, table, lens, 8, q_offsets=offs)
    pd, qd, td, ld, od = dev(pools), q.to(DEV), table.to(DEV), lens.to(DEV), offs.to(DEV)
    size = ob.kvq_attention_workspace_bytes(5, q.shape[0], 8, 2, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(qd) for _ in range(8)] for _ in streams]
    wss = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for s, o, ws in zip(streams, outs, wss):
            ob.kvq_attention(qd, *pd, td, ld, o[i], bits=8, q_offsets=od, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for t in o:
            assert torch.equal(t.cpu(), want)


def test_binding_refusals_with_device_tensors():
    pools = dev(random_pools(2, 2, 16, 64, 8, gen("refuse")))
    q = torch.zeros(2, 4, 64, dtype=BF16, device=DEV)
    table, lens = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    ws = torch.zeros(ob.kvq_attention_workspace_bytes(2, 2, 4, 2, 64), dtype=torch.uint8, device=DEV)
    ok = dict(q=q, table=table, lens=lens, out=torch.zeros_like(q), kw=dict(bits=8, workspace=ws))

    def call(**kw):
        a = {**ok, **kw}
        ob.kvq_attention(a["q"], *pools, a["table"], a["lens"], a["out"], **{**ok["kw"], **a["kw"]})

    call()
    for bad, kw in [
        (ValueError, dict(q=q[:, :, :32])), (ValueError, dict(q=q[0])), (ValueError, dict(out=q[:1])),
        (ValueError, dict(out=q.float())), (ValueError, dict(lens=lens[:1])), (TypeError, dict(lens=lens.long())),
        (TypeError, dict(table=table.long())), (ValueError, dict(table=table[0])), (TypeError, dict(lens=lens.cpu())),
        (TypeError, dict(kw=dict(q_offsets=torch.zeros(3, device=DEV)))),
        (ValueError, dict(kw=dict(q_offsets=torch.zeros(2, dtype=torch.int32, device=DEV)))),
        (ValueError, dict(kw=dict(lse=torch.zeros(2, 2, device=DEV)))),
        (ob.OnebitError, dict(kw=dict(window=-1))), (ob.OnebitError, dict(kw=dict(softcap=-1.0))),
        (ValueError, dict(kw=dict(window=2 ** 32 + 1))), (ValueError, dict(kw=dict(workspace=ws[:64].expand(ws.numel(), 64)))),
        (ob.OnebitError, dict(kw=dict(workspace=ws[:16]))), (ob.OnebitError, dict(q=q.float(), out=q.float())),
        (ob.OnebitError, dict(q=torch.zeros(2, 3, 64, dtype=BF16, device=DEV),
                              out=torch.zeros(2, 3, 64, dtype=BF16, device=DEV))),
    ]:
        with pytest.raises(bad):
            call(**kw)
    k = torch.zeros(2, 2, 64, dtype=BF16, device=DEV)
    at = torch.tensor([0, 1], device=DEV)
    for bad, args in [(ValueError, (k, k.float(), at)), (ValueError, (k, k[:1], at)), (TypeError, (k, k, at.int())),
                      (ValueError, (k, k, at[:1])), (TypeError, (k.double(), k.double(), at)),
                      (ob.OnebitError, (torch.zeros(2, 2, 65, dtype=BF16, device=DEV)[:, :, :64],) * 2 + (at,))]:
        with pytest.raises(bad):
            ob.kvq_quantize(*args, *pools, bits=8)
    with pytest.raises(ValueError):
        ob.kvq_dequantize(*pools, at, k.transpose(0, 1), k, bits=8)
