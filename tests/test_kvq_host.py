"""The coded cache's calls refuse what they cannot serve before anything is launched
(no GPU needed), and the tests' own 64-bit reference is pinned."""
import ctypes as C
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import kvq_ref
from error_compensated_bit_amd import onebit as ob

INV, ALIGN, UNSUP, OK = (ob.ONEBIT_ERR_INVALID, ob.ONEBIT_ERR_ALIGN, ob.ONEBIT_ERR_UNSUPPORTED, ob.ONEBIT_OK)
A = 0x10000        # an address that is never touched: every call below is refused or empty


def cache(**kw):
    f = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, n_pages=4, page=16, kv_heads=2, head_dim=128, bits=8)
    f.update(kw)
    return ob.KvqCache(*[f[n] for n, _ in ob.KvqCache._fields_])


def write(c=None, k=A, v=A, dtype=ob.ONEBIT_BF16, tokens=3, st=(256, 128, 256, 128), slots=A):
    c = cache() if c is None else c
    return ob.load().kvq_quantize(k, v, dtype, tokens, *st, slots, C.byref(c), None)


def read(c=None, slots=A, tokens=3, k=A, v=A, dtype=ob.ONEBIT_BF16):
    c = cache() if c is None else c
    return ob.load().kvq_dequantize(C.byref(c), slots, tokens, k, v, dtype, None)


def attend(c=None, q=A, dtype=ob.ONEBIT_BF16, total=4, hq=4, qt=512, qh=128, offsets=None, kv=A, batch=2, table=A,
           max_pages=2, stride=2, scale=0.1, cap=0.0, window=0, out=A, lse=None, ws=A, ws_bytes=None):
    c = cache() if c is None else c
    if ws_bytes is None:
        ws_bytes = ob.kvq_attention_workspace_bytes(batch, total, hq, c.kv_heads, c.head_dim)
    return ob.load().kvq_attention(q, dtype, total, hq, qt, qh, offsets, kv, batch, table, max_pages, stride,
                                   C.byref(c), scale, cap, window, out, lse, ws, ws_bytes, None)


BAD_CACHES = [
    (dict(bits=5), INV), (dict(bits=0), INV), (dict(page=0), INV), (dict(page=8), INV), (dict(page=48), INV),
    (dict(page=2048), INV), (dict(page=-16), INV), (dict(kv_heads=0), INV), (dict(kv_heads=32768), INV),
    (dict(n_pages=-1), INV), (dict(n_pages=2 ** 43), INV), (dict(n_pages=2 ** 62), INV), (dict(head_dim=96), UNSUP),
    (dict(head_dim=0), UNSUP), (dict(head_dim=512), UNSUP), (dict(k_codes=None), INV), (dict(v_codes=None), INV),
    (dict(k_scales=None), INV), (dict(v_scales=None), INV), (dict(k_codes=A + 8), ALIGN), (dict(v_codes=A + 4), ALIGN),
    (dict(k_scales=A + 4), ALIGN), (dict(v_scales=A + 8), ALIGN),
]


@pytest.mark.parametrize("fields,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(fields, status):
    # the head counts of the attention call follow the cache's where they can
    heads = fields.get("kv_heads", 2)
    assert write(cache(**fields)) == status
    assert read(cache(**fields)) == status
    assert attend(cache(**fields), hq=4 if heads == 2 else max(heads, 1), ws_bytes=1 << 40) == status


def test_null_cache_is_refused():
    lib = ob.load()
    assert lib.kvq_quantize(A, A, 1, 3, 256, 128, 256, 128, A, None, None) == INV
    assert lib.kvq_dequantize(None, A, 3, A, A, 1, None) == INV
    assert lib.kvq_attention(A, 1, 4, 4, 512, 128, None, A, 2, A, 2, 2, None, 0.1, 0.0, 0, A, None, A, 1 << 30,
                             None) == INV


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(tokens=-1), INV), (dict(tokens=1 << 26), INV),
    (dict(k=None), INV), (dict(v=None), INV), (dict(slots=None), INV), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN),
    (dict(slots=A + 4), ALIGN), (dict(st=(260, 128, 256, 128)), ALIGN), (dict(st=(256, 129, 256, 128)), ALIGN),
    (dict(st=(256, 128, 4, 128)), ALIGN), (dict(st=(256, 128, 256, 2)), ALIGN),
    (dict(dtype=ob.ONEBIT_F32, st=(256, 128, 256, 2)), ALIGN),
    (dict(tokens=0, k=None, v=None, slots=None), OK),
])
def test_write_refusals(kw, status):
    assert write(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INV), (dict(tokens=-1), INV), (dict(tokens=1 << 26), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(slots=None), INV), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(slots=A + 4), ALIGN),
    (dict(tokens=0, k=None, v=None, slots=None), OK),
])
def test_read_refusals(kw, status):
    assert read(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=ob.ONEBIT_F32), UNSUP), (dict(dtype=7), INV), (dict(total=-1, ws_bytes=1 << 30), INV),
    (dict(hq=3, ws_bytes=1 << 30), INV), (dict(hq=0, ws_bytes=1 << 30), INV), (dict(hq=1, ws_bytes=1 << 30), INV),
    (dict(batch=-1, ws_bytes=1 << 30), INV), (dict(batch=3), INV),        # 4 rows are no multiple of 3
    (dict(total=2 ** 31, hq=2, ws_bytes=1 << 40), INV), (dict(total=2 ** 30, ws_bytes=1 << 40), INV),
    (dict(max_pages=-1), INV), (dict(max_pages=2 ** 27), INV), (dict(max_pages=3), INV),   # rows closer than 3
    (dict(window=-1), INV), (dict(cap=-1.0), INV), (dict(cap=math.nan), INV), (dict(cap=math.inf), INV),
    (dict(cap=2.0 ** 65), INV), (dict(cap=2.0 ** -65), INV), (dict(scale=-2.0 ** 65), INV),
    (dict(cap=1e39), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(scale=1e39), INV),
    (dict(q=None), INV), (dict(kv=None), INV), (dict(out=None), INV), (dict(table=None), INV), (dict(ws=None), INV),
    (dict(ws_bytes=0), INV), (dict(q=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(ws=A + 8), ALIGN),
    (dict(qt=516), ALIGN), (dict(qh=4), ALIGN), (dict(kv=A + 2), ALIGN), (dict(table=A + 2), ALIGN),
    (dict(offsets=A + 1), ALIGN), (dict(lse=A + 2), ALIGN),
    (dict(batch=0, q=None, kv=None, out=None, ws=None, table=None), OK),
    (dict(total=0, q=None, kv=None, out=None, ws=None, table=None), OK),
])
def test_attention_refusals(kw, status):
    assert attend(**kw) == status


def test_workspace_size_is_zero_for_refused_sizes_and_enough_is_asked_for():
    f = ob.kvq_attention_workspace_bytes
    assert f(2, 4, 4, 2, 128) > 0 and f(1, 1, 1, 1, 64) > 0 and f(0, 0, 1, 1, 64) > 0
    for bad in [(-1, 4, 4, 2, 128), (2, -4, 4, 2, 128), (2, 4, 3, 2, 128), (2, 4, 0, 2, 128), (2, 4, 4, 0, 128),
                (2, 4, 4, 2, 96), (2, 2 ** 31, 4, 2, 128), (2 ** 26, 4, 4, 2, 128), (2 ** 62, 4, 4, 2, 128)]:
        assert f(*bad) == 0, bad
    need = f(2, 4, 4, 2, 128)
    assert attend(ws_bytes=need - 1) == INV


def test_binding_refuses_host_and_mismatched_tensors():
    """Nothing below reaches the library: host tensors are refused first."""
    codes = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    scales = torch.zeros(4, 2, 16)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.arange(3)
    pools = (codes, scales, codes.clone(), scales.clone())
    with pytest.raises(TypeError):
        ob.kvq_quantize(k, k.clone(), slots, *pools, bits=8)
    with pytest.raises(TypeError):
        ob.kvq_dequantize(*pools, slots, k, k.clone(), bits=8)
    with pytest.raises(TypeError):
        ob.kvq_attention(k, *pools, torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32),
                         torch.zeros_like(k), bits=8, workspace=torch.zeros(32, dtype=torch.int64))


@pytest.mark.parametrize("bad,kw", [
    (ValueError, dict(bits=3)), (ValueError, dict(v_codes=torch.zeros(4, 2, 16, 64, dtype=torch.uint8))),
    (ValueError, dict(k_scales=torch.zeros(4, 2, 8))), (TypeError, dict(k_codes=torch.zeros(4, 2, 16, 128))),
    (TypeError, dict(v_scales=torch.zeros(4, 2, 16, dtype=torch.float64))),
    (ValueError, dict(k_codes=torch.zeros(4, 16, 2, 128, dtype=torch.uint8).transpose(1, 2))),
    (ValueError, dict(k_codes=torch.zeros(2, 16, 128, dtype=torch.uint8))),
])
def test_binding_checks_the_cache_tensors(bad, kw):
    base = dict(k_codes=torch.zeros(4, 2, 16, 128, dtype=torch.uint8), k_scales=torch.zeros(4, 2, 16),
                v_codes=torch.zeros(4, 2, 16, 128, dtype=torch.uint8), v_scales=torch.zeros(4, 2, 16), bits=8)
    c = ob._kvq_cache(**base)
    assert (c.n_pages, c.kv_heads, c.page, c.head_dim, c.bits) == (4, 2, 16, 128, 8)
    with pytest.raises(bad):
        ob._kvq_cache(**{**base, **kw})


def test_binding_takes_the_strides_of_row_tensors():
    wide = torch.zeros(5, 7, 64)
    assert ob._kvq_rows(wide[:, 2:4], 2, 64, "k") == (7 * 64, 64)
    assert ob._kvq_rows(wide.transpose(0, 1), 5, 64, "k") == (64, 7 * 64)
    assert ob._kvq_rows(wide[:1, :1], 1, 64, "k") == (64, 64)            # unused strides are replaced
    with pytest.raises(ValueError):
        ob._kvq_rows(wide, 6, 64, "k")
    with pytest.raises(ValueError):
        ob._kvq_rows(torch.zeros(5, 64, 7).transpose(1, 2), 7, 64, "k")


@pytest.mark.parametrize("bits", [4, 8])
def test_reference_codes_against_fractions(bits):
    """The reference's codes are the exact quotients' nearest integers (ties to even) for the
    stored reciprocal, and a value is off by at most half a step (and the reciprocal's rounding)."""
    top, z = kvq_ref.LEVELS[bits]
    rng = np.random.default_rng(bits)
    x = torch.from_numpy(rng.standard_normal((40, 64)).astype(np.float32)).to(torch.bfloat16)
    x[0] = torch.arange(64) * 0.5 - 16.0                                  # ties where amax = L (below)
    x[0, 0] = top
    x[1] = 0.0
    codes, scales = kvq_ref.code_rows(x, bits)
    for r in range(40):
        row = [Fraction(float(t)) for t in x[r]]
        amax = max(abs(t) for t in row)
        if amax == 0:
            assert scales[r] == 0 and (codes[r] == z).all()
            continue
        inv = Fraction(float(np.float32(top) / np.float32(float(amax))))
        scale = np.float32(float(amax)) / np.float32(top)
        assert float(scales[r]) == float(scale)
        for t, c in zip(row, codes[r].tolist()):
            assert c == round(t * inv) + z                                # round() of a Fraction: ties to even
            assert abs((c - z) * Fraction(float(scale)) - t) <= Fraction(float(scale)) * Fraction(50001, 100000)


def test_reference_pack_round_trip():
    code = torch.randint(0, 16, (3, 5, 64), dtype=torch.uint8)
    assert torch.equal(kvq_ref.unpack(kvq_ref.pack(code, 4), 4), code)
    assert kvq_ref.pack(code, 4)[0, 0, 0] == code[0, 0, 0] + 16 * code[0, 0, 1]
