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


def rows_keep_their_bits(q_len, kv, dtype, bits, dim, junk, window, pages=0):
    """Tokens of the new ones from the middle on, then those in front of the last queries' windows, hold
    other values: queries that do not attend to them keep their bits, and the others are right."""
    g = gen("later", q_len, kv, dim, bits)
    q, pools, table, lens, _ = make(g, [q_len, q_len], [kv, kv + 37], 4, 2, dim, 16, bits, dtype)
    if pages > table.shape[1]:
        table = torch.cat((table, torch.full((2, pages - table.shape[1]), -1, dtype=torch.int32)), 1)
    kw = dict(window=window)
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
