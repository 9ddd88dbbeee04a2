"""How much workspace the products with coded weights ask for (no GPU needed)."""
import pytest

from error_compensated_bit_amd import onebit as ob
from test_qsdp_linear_host import ALIGN, INV, matrix, product

SIZE = ob.qsdp_linear_workspace_bytes
FEW = ob.QSDP_LINEAR_EXACT_TOKENS


@pytest.mark.parametrize("rows,cols", [(50257, 1600), (28672, 8192), (1, 32)])
def test_few_tokens_are_sized_by_the_gradient(rows, cols):
    """qsdp_linear with few tokens has no partial results."""
    for tokens in (1, 7, FEW):
        assert SIZE(tokens, rows, cols) == SIZE(tokens, 1, cols)
    assert SIZE(FEW + 1, rows, cols) == max(SIZE(FEW + 1, rows, 32), SIZE(FEW + 1, 1, cols))


@pytest.mark.parametrize("rows,cols", [(50257, 1600), (96, 64), (6400, 1600), (1, 4096), (4096, 32)])
def test_no_fewer_bytes_with_more_tokens(rows, cols):
    sizes = [SIZE(t, rows, cols) for t in (*range(0, 300), 511, 512, 513, 4096, 50000, (1 << 24) - 1)]
    assert sizes == sorted(sizes) and sizes[0] >= 16


def test_what_a_call_refuses():
    """Each direction by its own result."""
    w = matrix(rows=50257, cols=64)
    for tokens in (1, FEW):
        assert product("qsdp_linear", w, tokens=tokens, os=60000, ws_bytes=15) == INV
        assert product("qsdp_linear", w, tokens=tokens, os=60000, ws_bytes=16, ws=0x10008) == ALIGN
        assert product("qsdp_linear", w, tokens=tokens, os=60000, ws_bytes=16, ws=None) == INV
    # one byte short: the other operand's size does not help
    assert product("qsdp_linear", w, tokens=FEW + 1, os=60000, ws_bytes=SIZE(FEW + 1, 50257, 32) - 1) == INV
    assert product("qsdp_linear_grad", w, tokens=3, xs=60000, ws_bytes=SIZE(3, 1, 64) - 1) == INV
