"""Where lanes of a wave read what others wrote, or write what others have read, without a workgroup's
barrier, a wave barrier holds the order: to the compiler the addresses of one lane need not be those of
another, so nothing else keeps its loads and stores apart.  Read from the kernels' own assembly."""
import os
import re
import shutil
import subprocess

import pytest

from error_compensated_bit_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


def kernels(name, *defines):
    """Instructions and wave barriers of each kernel in the order of the listing."""
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc is not installed")
    flags = [f for f in build.command("x")[1:-2] if not f.endswith(".hip") and f not in ("-shared", "-fPIC")]
    text = subprocess.run(["hipcc", *flags, *defines, "--offload-device-only", "-S", os.path.join(HERE, "wave_exchange.hip"),
                           "-o", "-"], check=True, capture_output=True, text=True).stdout
    for body in re.findall(r"^(_ZN6onebit\w*%s\w*):.*?\n(.*?)^\.Lfunc_end" % name, text, re.M | re.S):
        yield body[0], [m.group(0) for m in re.finditer(r"; wave barrier|\b[a-z][a-z0-9_]+\b(?=\s)", body[1])]


def unfenced(listing):
    """Reads of LDS with a write in front of them and no barrier between."""
    written, found = False, 0
    for op in listing:
        if op in ("s_barrier", "; wave barrier"):
            written = False
        elif op.startswith("ds_write"):
            written = True
        elif op.startswith("ds_read"):
            found += written
    return found


def test_codes_turned_through_lds():
    seen = 0
    for name, listing in kernels("k_qsdp_rows", "-DROWS"):
        assert sum(op.startswith("ds_read") for op in listing) and sum(op.startswith("ds_write") for op in listing), name
        assert unfenced(listing) == 0, name
        seen += 1
    assert seen == 2


def test_queries_turned_in_place():
    """All of a row is read before any of it is written."""
    seen = 0
    for name, listing in kernels("k_kvq_append"):
        if "ILi1ELi128ELi8E" not in name:
            continue
        stores = [i for i, op in enumerate(listing) if op.startswith("global_store")]
        loads = [i for i, op in enumerate(listing) if op.startswith("global_load")]
        fences = [i for i, op in enumerate(listing) if op == "; wave barrier"]
        assert stores and loads and max(loads) < min(stores), name
        assert any(max(loads) < i < min(stores) for i in fences), name
        seen += 1
    assert seen == 1


def test_the_check_itself():
    assert unfenced(["ds_write_b128", "ds_read_b128", "ds_read_b128"]) == 2
    assert unfenced(["ds_write_b128", "; wave barrier", "ds_read_b128", "s_barrier", "ds_read_b32"]) == 0
