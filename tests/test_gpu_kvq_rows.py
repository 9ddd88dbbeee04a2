"""kvq_attention on the GPU, row by row: a query's result depends on nothing but the
tokens it attends to itself, whatever the scales of those are."""
import math

import pytest
import torch

import kvq_ref
from test_gpu_kvq import attend, check, gen, make

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def rows_of(pools, table, b, positions):
    """(pages, offsets) of a sequence's positions."""
    page = pools[0].shape[2]
    at = torch.as_tensor(list(positions), dtype=torch.long)
    return table[b].long()[at // page], at % page


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("softcap", [0.0, 5.0, 100.0])
@pytest.mark.parametrize("q_len,kv,at", [(1, 90, 40), (5, 90, 87), (70, 100, 83), (300, 300, 140)])
@pytest.mark.parametrize("which,bad", [(1, math.inf), (1, -math.inf), (1, math.nan), (3, -math.inf), (3, math.inf)])
def test_no_scale_that_is_not_finite_leaves_a_finite_output(dtype, softcap, q_len, kv, at, which, bad):
    """Keys of an infinite scale, whatever the sign of their products with the query and with a cap
    above them: as with any scale that is not finite, nothing finite for those who attend to the row."""
    g = gen("infinite", q_len)
    q, pools, table, lens, offs = make(g, [q_len], [kv], 4, 2, 64, 16, 8, dtype)
    ref = kvq_ref.attention(q, pools, table, lens, bits=8, scale=0.125, softcap=softcap)
    dirty = [p.clone() for p in pools]
    page, offset = rows_of(pools, table, 0, [at])
    dirty[which][page, :, offset] = bad
    got, _ = attend(q, tuple(dirty), table, lens, 8, softcap=softcap)
    first = max(0, at - (kv - q_len))               # the first query that attends to the row
    assert not torch.isfinite(got[first:]).any()
    check(got[:first], None, tuple(t[:first] for t in ref), dtype)


JUNK = [2.0 ** 20, 2.0 ** 100, -2.0 ** 120, math.inf, math.nan, 2.0 ** -110]


def spoil(pools, table, b, positions, junk, g):
    """The cache with rows of a sequence replaced: codes at random, scales of `junk` with either sign."""
    out = [p.clone() for p in pools]
    pages, offsets = rows_of(pools, table, b, positions)
    for which in (0, 2):
        codes = out[which][pages, :, offsets]
        out[which][pages, :, offsets] = torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8)
        sign = torch.randint(0, 2, out[which + 1][pages, :, offsets].shape, generator=g).float() * 2 - 1
        out[which + 1][pages, :, offsets] = sign * junk
    return tuple(out)


def rows_keep_their_bits(q_len, kv, dtype, bits, dim, junk, window, pages=0, softcap=0.0, group=2):
    """Tokens of the new ones from the middle on, then those in front of the last queries' windows, hold
    other values: queries that do not attend to them keep their bits."""
    g = gen("later", q_len, kv, dim, bits)
    q, pools, table, lens, _ = make(g, [q_len, q_len], [kv, kv + 37], 2 * group, 2, dim, 16, bits, dtype)
    if pages > table.shape[1]:
        table = torch.cat((table, torch.full((2, pages - table.shape[1]), -1, dtype=torch.int32)), 1)
    kw = dict(window=window, softcap=softcap)
    want, want_lse = attend(q, pools, table, lens, bits, **kw)
    for b in range(2):
        n = int(lens[b])
        start = n - q_len                               # the first query's position
        own = slice(b * q_len, (b + 1) * q_len)
        cut = q_len // 2
        got, lse = attend(q, spoil(pools, table, b, range(start + cut, n), junk, g), table, lens, bits, **kw)
        assert torch.equal(got[own][:cut], want[own][:cut]) and torch.equal(lse[own][:cut], want_lse[own][:cut])
        other = slice((1 - b) * q_len, (2 - b) * q_len)
        assert torch.equal(got[other], want[other])
        if window:
            front = range(0, max(0, start + cut - window + 1))    # queries from `cut` on do not reach these
            got, lse = attend(q, spoil(pools, table, b, front, junk, g), table, lens, bits, **kw)
            assert torch.equal(got[own][cut:], want[own][cut:]) and torch.equal(lse[own][cut:], want_lse[own][cut:])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits,dim", [(8, 128), (4, 64), (8, 256)])
@pytest.mark.parametrize("q_len,kv,pages", [(8, 8, 0), (8, 700, 0), (24, 24, 0), (24, 300, 0), (12, 300, 70000)])
@pytest.mark.parametrize("junk", JUNK)
@pytest.mark.parametrize("window", [0, 5, 90])
def test_drafts_know_nothing_of_later_tokens(dtype, bits, dim, q_len, kv, pages, junk, window):
    """Blocks of 16 rows (tokens x 2), and of 32 under a block table for long caches."""
    rows_keep_their_bits(q_len, kv, dtype, bits, dim, junk, window, pages)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits,dim", [(8, 128), (4, 64), (8, 256), (4, 128)])
@pytest.mark.parametrize("q_len,kv", [(60, 400), (300, 300)])
@pytest.mark.parametrize("size", [3.0, 30.0, 300.0])
def test_large_scores_of_chunks_are_as_exact_as_binary32(dtype, bits, dim, q_len, kv, size):
    """Scores of about `size`, all sums of terms of one sign.  What a score may be off by is then a part
    of itself: the products' sum in binary32, at most a rounding of 2^-24 for each of D terms (taken
    twice, the matrix cores may cut where others round), the two scales' roundings, and exp2's argument,
    2^-22 (s + 1).  lse is off by as much and by its sum's roundings; an output by twice as much of
    A = sum_j softmax_j |v_j| (the weights and their sum), by the weights' rounding to fp16, 2^-11 A, for
    bf16 by that of the values and their scales, 2^-10 A + 2^-14 of the largest scale, by its sums, and
    by its own rounding."""
    g = gen("large", q_len, dim, bits)
    q, pools, table, lens, _ = make(g, [q_len], [kv], 4, 2, dim, 16, bits, dtype)
    zero = kvq_ref.LEVELS[bits][1]
    code = kvq_ref.unpack(pools[0], bits)
    pools = (kvq_ref.pack(torch.where(code < zero, 2 * zero - code, code), bits), *pools[1:])
    q = q.abs()
    pages, offsets = rows_of(pools, table, 0, range(kv))
    k, v = (kvq_ref.values(pools[i][pages, :, offsets], pools[i + 1][pages, :, offsets], bits) for i in (0, 2))
    x = q.double().view(q_len, 2, 2, dim)
    raw = torch.einsum("tghd,jgd->tghj", x, k)
    scale = size / float(raw.mean())
    late = (torch.arange(kv) > torch.arange(kv - q_len, kv).unsqueeze(1)).view(q_len, 1, 1, kv)
    s = (scale * raw).masked_fill(late, -math.inf)
    want_lse = torch.logsumexp(s, -1)
    p = torch.softmax(s, -1)
    want, a = (torch.einsum("tghj,jgd->tghd", p, t) for t in (v, v.abs()))
    top = s.amax(-1)
    off = 2 * (dim + 8) * 2.0 ** -24 * top + 2.0 ** -22 * (top + 1)
    sums = 2.0 ** -24 * (kv + 64)
    v_top = float(pools[3][pages, :, offsets].abs().max())
    tol = a * (2 * off.unsqueeze(-1) + 2.0 ** -11 + 4 * sums) + 2.0 ** -20 * v_top
    if dtype == BF16:
        tol = tol + 2.0 ** -10 * a + 2.0 ** -14 * v_top
    tol = tol + kvq_ref.HALF_STEP[dtype] * (want.abs() + tol)
    got, lse = attend(q, pools, table, lens, bits, scale=scale)
    assert ((lse.double().view_as(want_lse) - want_lse).abs() <= off + sums + 2.0 ** -22 * (want_lse.abs() + 1)).all()
    assert ((got.double().view_as(want) - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("q_len", [5, 70])
@pytest.mark.parametrize("key_exp,scale_exp", [(118, -121), (118, -110), (118, None), (-110, 64), (100, None), (90, -100)])
@pytest.mark.parametrize("window", [0, 30])
def test_keys_of_any_size_with_a_scale_that_brings_the_scores_back(dtype, bits, q_len, key_exp, scale_exp, window):
    """Keys near binary32's ends, and a scale of the scores of 0 (None)."""
    g = gen("keys", q_len, bits)
    q, pools, table, lens, offs = make(g, [q_len] * 2, [200, 300], 4, 2, 256, 16, bits, dtype, peaked=0.5)
    pools[1].mul_(2.0 ** key_exp)
    scale = 0.0 if scale_exp is None else 2.0 ** scale_exp
    if scale_exp is not None:       # queries that make the scores of some size
        q = (q.double() * 2.0 ** max(-8, min(8, -key_exp - scale_exp))).to(dtype)
    got, lse = attend(q, pools, table, lens, bits, q_offsets=offs, scale=scale, window=window)
    ref = kvq_ref.attention(q, pools, table, lens, bits=bits, scale=scale, q_offsets=offs, window=window)
    check(got, lse, ref, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits,dim", [(8, 128), (4, 64), (8, 256)])
@pytest.mark.parametrize("q_len,kv", [(70, 70), (70, 900), (300, 333)])
@pytest.mark.parametrize("junk", JUNK)
@pytest.mark.parametrize("window", [0, 40, 200])
def test_chunks_know_nothing_of_later_tokens(dtype, bits, dim, q_len, kv, junk, window):
    rows_keep_their_bits(q_len, kv, dtype, bits, dim, junk, window)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_len,kv", [(24, 300), (70, 333)])
@pytest.mark.parametrize("softcap", [4.0, 100.0])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("junk", [2.0 ** 100, math.inf])
def test_later_tokens_under_a_cap(dtype, q_len, kv, softcap, window, junk):
    rows_keep_their_bits(q_len, kv, dtype, 8, 128, junk, window, softcap=softcap)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_later_tokens_with_more_heads_of_a_cache_head_than_a_tile_has_rows(dtype):
    rows_keep_their_bits(6, 90, dtype, 8, 64, 2.0 ** 100, 20, group=300)


def values_without_sign(codes):
    """Codes (8 bits) of the magnitudes of the values."""
    return torch.where(codes < 128, (256 - codes.int()).clamp(max=255).to(torch.uint8), codes)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_len,kv,dim", [(24, 60, 128), (70, 70, 128), (300, 340, 128), (200, 900, 64), (150, 700, 256)])
@pytest.mark.parametrize("step", [3.0, 0.25, -0.25, -3.0])
@pytest.mark.parametrize("window", [0, 300])
def test_scales_that_change_along_the_tokens(dtype, q_len, kv, dim, step, window):
    """Every token's values are 2^step times the last one's (from 2^-90 to 2^90 where they would go
    further).  A query's tolerance counts its own tokens only: it is computed for the cache that ends with
    it, and for bf16 allows for the values' rounding in chunks, 2^-10 A and 2^-14 of the largest scale."""
    g = gen("change", q_len)
    q, pools, table, lens, _ = make(g, [q_len], [kv], 4, 2, dim, 16, 8, dtype, spread=False)
    pages, offsets = rows_of(pools, table, 0, range(kv))
    size = torch.exp2(((torch.arange(kv) - (kv - q_len // 2)) * step).clamp(-90, 90).round())
    if dtype == F16:
        size = size.clamp(2.0 ** -14, 2.0 ** 8)              # (what the output can hold)
    pools[3][pages, :, offsets] *= size.unsqueeze(1)
    magnitudes = (*pools[:2], values_without_sign(pools[2]), pools[3])
    kw = dict(bits=8, scale=dim ** -0.5, window=window)
    got, lse = attend(q, pools, table, lens, **kw)
    for t in sorted({0, 1, 7, 8, q_len // 3, q_len // 2, q_len - 2, q_len - 1}):
        n = kv - q_len + t + 1                               # tokens up to the query's own
        ref = kvq_ref.attention(q[t:t + 1], pools, table, torch.tensor([n]), **kw)
        first = max(0, n - window) if window else 0
        own = float(pools[3][pages[first:n], :, offsets[first:n]].max())
        a = kvq_ref.attention(q[t:t + 1], magnitudes, table, torch.tensor([n]), **kw)[0]
        tol = ref[2] + (2.0 ** -10 * a + 2.0 ** -14 * own if dtype == BF16 else 0.0)
        check(got[t:t + 1], lse[t:t + 1], (ref[0], ref[1], tol, ref[3], ref[4]), dtype)
