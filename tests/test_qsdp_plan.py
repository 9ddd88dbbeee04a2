"""How the tiled products with coded weights are cut up (host code of the library's header, compiled
and run here), and what the GPU tests' tolerance can see."""
import ctypes as C
import math
import os
import random
import shutil
import subprocess

import pytest
import torch

import qsdp_linear_ref as ref
import qsdp_tile_ref as tiles
from error_compensated_bit_amd import onebit as ob

HERE = os.path.dirname(os.path.abspath(__file__))
DEPTH = 64          # of a step


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    out = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(os.path.dirname(HERE), "error_compensated_bit_amd", "csrc"),
                    os.path.join(HERE, "qsdp_plan_driver.cpp"), "-o", out], check=True, capture_output=True)
    call = C.CDLL(out).qsdp_plan
    call.argtypes, call.restype = [C.c_int64] * 3 + [C.c_int, C.c_void_p], None

    def run(op, tokens, rows, cols):
        """(tile, tiles along the tokens, along the result's columns, shares, tokens and columns of a tile)"""
        p = (C.c_int64 * 6)()
        call(tokens, *((rows, cols, 0) if op == "linear" else (cols, rows, 1)), p)
        return tuple(p)
    return run


def sizes(n):
    rng = random.Random(11)

    def size(most):
        return max(1, min(most, round(math.exp(rng.uniform(0.0, math.log(most))))))
    for _ in range(n):
        yield size(1 << rng.randint(1, 24)) % (1 << 24) or 1, size((1 << 24) - 1), 32 * size((1 << 19) - 1)
        yield size(9000), size(60000), 32 * size(512)


def test_every_plan_fits_its_workspace(plan):
    chosen = set()
    for tokens, rows, cols in sizes(4000):
        for op in ("linear", "grad"):
            if op == "linear" and tokens <= ob.QSDP_LINEAR_EXACT_TOKENS:
                continue
            shape, m, n, splits, tm, tn = plan(op, tokens, rows, cols)
            width, depth = (rows, cols) if op == "linear" else (cols, rows)
            assert 0 <= shape < 4 and m == -(-tokens // tm) and n == -(-width // tn)
            assert 1 <= splits <= min(16, -(-depth // DEPTH))
            need = ob.qsdp_linear_workspace_bytes(tokens, *((rows, 32) if op == "linear" else (1, cols)))
            assert splits == 1 or m * n * splits * tm * tn * 4 <= need, (op, tokens, rows, cols)
            chosen.add((op, shape, splits))
    # every tile is chosen by some size, alone and with its depth shared
    for op in ("linear", "grad"):
        for shape in range(4):
            assert (op, shape, 1) in chosen and {s for o, k, s in chosen if (o, k) == (op, shape)} >= {2, 3, 4, 6, 8, 12, 16}


@pytest.mark.parametrize("op,tokens,rows,cols,shape,splits", tiles.PLANNED)
def test_sizes_that_the_gpu_tests_rely_on(plan, op, tokens, rows, cols, shape, splits):
    """Where another plan is chosen for one of these, the list needs another size for this one."""
    got = plan(op, tokens, rows, cols)
    assert (got[0], got[3]) == (shape, splits)


def test_the_gpu_tests_sizes_reach_every_tile():
    have = {(op, shape, splits > 1) for op, _, _, _, shape, splits in tiles.PLANNED}
    # (the largest tile alone, forward, is what the tests of many tokens take)
    assert have >= {(op, s, shared) for op in ("linear", "grad") for s in range(4) for shared in (False, True)} - {("linear", 0, False)}


@pytest.mark.parametrize("op,tokens,rows,cols", [("grad", 40, 50257, 32), ("grad", 1, 20011, 96), ("linear", 70, 40, 12000),
                                                 ("grad", 130, 8192, 64)])
@pytest.mark.parametrize("bits,bucket", [(4, 1024), (8, 96)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_tolerance_sees_a_step_left_out(op, tokens, rows, cols, bits, bucket, dtype):
    """One step of 64 missing from the sum: most results are off by more than the tolerance."""
    g = torch.Generator().manual_seed(rows + bits)
    w = tiles.tile_weights(*tiles.coded_weights(rows, cols, bucket, bits, g), rows, cols, bucket, bits, dtype)
    depth = cols if op == "linear" else rows
    x = torch.randn(tokens, depth, generator=g).to(dtype)
    y, tol = tiles.tile_product(op, x, w)
    at = depth // 128 * 64
    short = x.clone()
    short[:, at:at + DEPTH] = 0
    off = (tiles.tile_product(op, short, w)[0] - y).abs() / tol
    assert (off > 1.0).double().mean() > 0.5
    # and the product's own rounding stays inside
    assert torch.all((y.to(dtype).double() - y).abs() <= tol)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rounded_weights_are_within_half_a_step(bits, dtype):
    g = torch.Generator().manual_seed(bits)
    coded = tiles.coded_weights(70, 96, 64, bits, g)
    w, _ = ref.weights(*coded, 70, 96, 64, bits)
    r = tiles.tile_weights(*coded, 70, 96, 64, bits, dtype)
    half = ref.HALF_STEP[dtype]
    # (rounded to fp32 first: half a step of that more; fp16 below 2^-14 is held to 2^-25)
    assert torch.all((r - w).abs() <= (half + 2.0 ** -24) * w.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0))
