"""The products with coded weights refuse what they cannot serve before anything is launched
(no GPU needed), and the tests' own 64-bit reference is pinned."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
import qsdp_linear_ref as ref
from error_compensated_bit_amd import onebit as ob

INV, ALIGN, UNSUP, OK = (ob.ONEBIT_ERR_INVALID, ob.ONEBIT_ERR_ALIGN, ob.ONEBIT_ERR_UNSUPPORTED, ob.ONEBIT_OK)
A = 0x10000        # an address that is never touched: every call below is refused or empty
NAMES = ("qsdp_linear", "qsdp_linear_grad")


def matrix(**kw):
    f = dict(codes=A, bucket_min=A, bucket_max=A, rows=96, cols=64, bucket=128, bits=4)
    f.update(kw)
    return ob.QsdpMatrix(*[f[n] for n, _ in ob.QsdpMatrix._fields_])


def product(name, w=None, x=A, dtype=ob.ONEBIT_BF16, tokens=3, xs=128, out=A, os=128, ws=A, ws_bytes=1 << 40):
    w = matrix() if w is None else w
    return getattr(ob.load(), name)(x, dtype, tokens, xs, C.byref(w), out, os, ws, ws_bytes, None)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("fields,status", [
    (dict(bits=5), INV), (dict(bits=0), INV), (dict(bucket=0), INV), (dict(bucket=-32), INV), (dict(bucket=65568), INV),
    (dict(bucket=16), UNSUP), (dict(bucket=100), UNSUP), (dict(rows=0), INV), (dict(rows=-1), INV),
    (dict(rows=1 << 24), INV), (dict(rows=2 ** 62), INV), (dict(cols=0), INV), (dict(cols=-32), INV),
    (dict(cols=1 << 24), INV), (dict(cols=33), UNSUP), (dict(cols=16), UNSUP), (dict(codes=None), INV),
    (dict(bucket_min=None), INV), (dict(bucket_max=None), INV), (dict(codes=A + 8), ALIGN),
    (dict(bucket_min=A + 2), ALIGN), (dict(bucket_max=A + 1), ALIGN),
])
def test_bad_matrices_are_refused(name, fields, status):
    assert product(name, matrix(**fields)) == status


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=ob.ONEBIT_F32), UNSUP), (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(tokens=-1), INV),
    (dict(tokens=1 << 24), INV), (dict(x=None), INV), (dict(out=None), INV), (dict(ws=None), INV), (dict(ws_bytes=0), INV),
    (dict(xs=56), INV), (dict(os=63), INV), (dict(xs=0), INV), (dict(xs=-128), INV), (dict(os=-128), INV),
    (dict(xs=1 << 23), INV), (dict(os=1 << 32), INV), (dict(xs=132), ALIGN), (dict(x=A + 8), ALIGN), (dict(out=A + 1), ALIGN),
    (dict(ws=A + 8), ALIGN), (dict(tokens=0, x=None, out=None, ws=None), OK),
])
def test_refusals(name, kw, status):
    assert product(name, **kw) == status


@pytest.mark.parametrize("name", NAMES)
def test_null_matrix_is_refused(name):
    assert getattr(ob.load(), name)(A, ob.ONEBIT_BF16, 3, 128, None, A, 128, A, 1 << 30, None) == INV


def test_a_workspace_one_byte_short_is_refused():
    need = ob.qsdp_linear_workspace_bytes(200, 96, 64)
    assert need >= 16
    for name in NAMES:
        assert product(name, tokens=200, ws_bytes=need - 1) == INV


@pytest.mark.parametrize("sizes", [(-1, 96, 64), (1 << 24, 96, 64), (4, 0, 64), (4, -3, 64), (4, 1 << 24, 64), (4, 96, 0),
                                   (4, 96, 48), (4, 96, 1 << 24), (4, 96, -32)])
def test_workspace_of_refused_sizes_is_zero(sizes):
    assert ob.qsdp_linear_workspace_bytes(*sizes) == 0


@pytest.mark.parametrize("sizes", [(0, 1, 32), (1, 1, 32), (64, 50257, 1600), (65, 100, 64), (4096, 1600, 6400),
                                   (1 << 23, 1, 32), ((1 << 24) - 1, (1 << 24) - 1, (1 << 24) - 32)])
def test_workspaces_stay_small(sizes):
    assert 16 <= ob.qsdp_linear_workspace_bytes(*sizes) <= 1 << 28


def test_host_tensors_and_mismatches_are_refused_by_the_binding():
    x, out = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, 96, dtype=torch.bfloat16)
    codes, lo = torch.zeros(96 * 32, dtype=torch.uint8), torch.zeros(48)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    with pytest.raises(TypeError):
        ob.qsdp_linear(x, codes, lo, lo, out, bucket=128, bits=4, workspace=ws)
    with pytest.raises(TypeError):
        ob.qsdp_linear_grad(out, codes, lo, lo, x, bucket=128, bits=4, workspace=ws)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,cols,bucket", [(3, 32, 32), (7, 96, 64), (5, 160, 1024), (9, 64, 96), (1, 4096, 4096)])
def test_reference_weights_are_the_oracles(bits, rows, cols, bucket):
    """The reference's weights against the framework's CPU oracle of the quantizer: half a step of fp32 for
    each of the oracle's two roundings."""
    n = rows * cols
    rng = np.random.default_rng(rows * cols + bits)
    x = torch.from_numpy((rng.standard_normal(n) * 0.02).astype(np.float32)).bfloat16()
    xb = x.view(torch.int16).numpy().view(np.uint16)
    codes, lo, hi = oracle.qsdp_quantize(xb, bucket=bucket, bits=bits, seed=5)
    _, y = oracle.qsdp_dequantize(codes, lo, hi, n, bucket=bucket, bits=bits, want_f32=True)
    t = [torch.from_numpy(np.array(a)) for a in (codes, lo, hi)]
    w, delta = ref.weights(*t, rows, cols, bucket, bits)
    y = torch.from_numpy(np.array(y)).double().view(rows, cols)
    scale = (2.0 ** bits) * delta + w.abs()
    assert torch.all((w - y).abs() <= 2.0 ** -24 * 2 * scale)


def test_reference_product_by_hand():
    """Two rows of 32: codes 0 .. 15 twice and 1 everywhere, minima -1 and 2, steps 0.5 and 0.25."""
    code = torch.cat((torch.arange(32) % 16, torch.ones(32, dtype=torch.int64))).to(torch.uint8)
    lo, hi = torch.tensor([-1.0, 2.0]), torch.tensor([-1.0 + 7.5, 2.0 + 3.75])
    w, delta = ref.weights(ref.pack(code, 4), lo, hi, 2, 32, 32, 4)
    assert w[0, 5] == -1.0 + 2.5 and w[1, 31] == 2.25 and delta[0, 0] == 0.5 and delta[1, 0] == 0.25
    y, tol = ref.product(torch.ones(1, 32), w.t(), delta.t(), 4, torch.bfloat16, True)
    assert y.tolist() == [[2 * (-16.0 + 0.5 * 120), 72.0]] and torch.all(tol > 0)
