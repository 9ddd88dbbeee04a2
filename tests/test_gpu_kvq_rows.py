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
