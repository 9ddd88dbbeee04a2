"""kvq_append refuses what it cannot serve before anything is launched (no GPU needed)."""
import ctypes as C

import pytest
import torch

from error_compensated_bit_amd import onebit as ob
from test_kvq_host import A, ALIGN, BAD_CACHES, INV, OK, cache


def append(c=None, q=A, k=A, v=A, dtype=ob.ONEBIT_BF16, tokens=3, heads=4, st=(512, 128, 256, 128, 256, 128), pos=A,
           rotary=A, far=100, rot=128, inter=0, slots=A, out=A, ot=512, oh=128):
    c = cache() if c is None else c
    return ob.load().kvq_append(q, k, v, dtype, tokens, heads, *st, pos, rotary, far, rot, inter, slots, C.byref(c), out,
                                ot, oh, None)


@pytest.mark.parametrize("fields,status", BAD_CACHES)
def test_bad_caches_are_refused(fields, status):
    assert append(cache(**fields), rot=16) == status


def strides(i, v):
    st = [512, 128, 256, 128, 256, 128]
    st[i] = v
    return tuple(st)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(tokens=-1), INV), (dict(tokens=1 << 26), INV),
    (dict(heads=-1), INV), (dict(heads=32768), INV), (dict(rot=0), INV), (dict(rot=8), INV), (dict(rot=24), INV),
    (dict(rot=144), INV), (dict(rot=-16), INV), (dict(far=0), INV), (dict(far=-1), INV), (dict(far=2 ** 41), INV),
    (dict(far=2 ** 62), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(out=None), INV),
    (dict(pos=None), INV), (dict(rotary=None), INV), (dict(slots=None), INV),
    (dict(q=A + 8), ALIGN), (dict(k=A + 2), ALIGN), (dict(v=A + 4), ALIGN), (dict(out=A + 8), ALIGN),
    (dict(rotary=A + 4), ALIGN), (dict(pos=A + 4), ALIGN), (dict(slots=A + 4), ALIGN), (dict(ot=513), ALIGN),
    (dict(oh=4), ALIGN), (dict(dtype=ob.ONEBIT_F32, oh=2), ALIGN), (dict(ot=516), ALIGN),
    *[(dict(st=strides(i, 4)), ALIGN) for i in range(6)], *[(dict(dtype=0, st=strides(i, 6)), ALIGN) for i in range(6)],
    (dict(tokens=0, q=None, k=None, v=None, pos=None, rotary=None, slots=None, out=None), OK),
])
def test_refusals(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("stride", [0, 64, 120, -120])
def test_rows_of_the_result_that_overlap_are_refused(stride):
    assert append(ot=stride) == INV
    assert append(oh=stride) == INV
    assert append(tokens=1, oh=stride) == INV


def test_null_cache_is_refused():
    assert ob.load().kvq_append(A, A, A, 1, 3, 4, 512, 128, 256, 128, 256, 128, A, A, 100, 128, 0, A, None, A, 512, 128,
                                None) == INV


def test_host_tensors_are_refused_by_the_binding():
    k, pools = torch.zeros(3, 2, 128), [torch.zeros(4, 2, 16, 128, dtype=torch.uint8), torch.zeros(4, 2, 16)] * 2
    i = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        ob.kvq_append(None, k, k, i, torch.zeros(9, 128), i, *pools, None, bits=8)
