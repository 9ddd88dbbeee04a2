"""The least workspace that the header names is enough, and nothing behind it is touched."""
import pytest
import torch

from error_compensated_bit_amd import onebit as ob
from test_gpu_qsdp_linear import BF16, DEV, EXACT, coded, dev, expect, gen, padded, run

pytestmark = pytest.mark.gpu
SIZE = ob.qsdp_linear_workspace_bytes


@pytest.mark.parametrize("op,tokens", [("linear", 1), ("linear", EXACT), ("linear", EXACT + 1), ("linear", 200),
                                       ("grad", 1), ("grad", EXACT), ("grad", 200)])
@pytest.mark.parametrize("rows,cols", [(5003, 160), (96, 4096)])
def test_least_workspace(op, tokens, rows, cols):
    bucket, bits = 1024, 4
    g = gen("least", op, tokens, rows)
    weights = dev(coded(rows, cols, bucket, bits, g, whole=True))
    x = torch.randint(-2, 3, (tokens, cols if op == "linear" else rows), generator=g).to(BF16)
    want = expect(op, x.to(DEV), weights, rows, cols, bucket, bits)[0].float().to(BF16)
    need = SIZE(tokens, 1, cols) if op == "grad" else 16 if tokens <= EXACT else SIZE(tokens, rows, 32)
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    got = run(op, padded(x), weights, rows, cols, bucket, bits, workspace=room[:need])
    assert torch.equal(got, want)
    assert torch.all(room[need:] == 0xA5)
    with pytest.raises(ob.OnebitError):
        run(op, padded(x), weights, rows, cols, bucket, bits, workspace=room[:need - 1])
