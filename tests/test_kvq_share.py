"""How kvq_attention's chunk kernel shares its work out: host code of the kernel's header, compiled
and run here."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc is not installed")
    out = str(tmp_path_factory.mktemp("share") / "driver")
    subprocess.run(["hipcc", "--offload-host-only", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "error_compensated_bit_amd", "csrc"), os.path.join(HERE, "kvq_share_driver.hip"),
                    "-o", out], check=True, capture_output=True)
    return out


@pytest.mark.parametrize("rows,tile", [(256, 128), (256, 64), (128, 32)])
@pytest.mark.parametrize("length,kv", [(64, 64), (700, 700), (4000, 4000), (4000, 9000), (2048, 34816), (513, 100000)])
@pytest.mark.parametrize("group", [1, 3, 4, 16])
@pytest.mark.parametrize("window", [0, 1, 200, 1024, 4096, 6000, 2 ** 31 - 1])
def test_a_row_tile_is_allotted_its_tiles(driver, rows, tile, length, kv, group, window):
    """Within two tiles (the bounds round to whole tiles at both ends) and a sixteenth for every row tile
    in front of it (the growth is held in sixteenths, cut), and the sums are those of the parts."""
    text = subprocess.run([driver, *map(str, (rows, tile, length, kv, group, window))], check=True, capture_output=True,
                          text=True).stdout.splitlines()
    setup, total = (int(x) for x in text[-1].split()[1:])
    assert len(text) - 1 == (-(-length * group // rows) if length * group > 48 else 0)
    at = 0
    for rt, line in enumerate(text[:-1]):
        share, tiles, before = (int(x) for x in line.split())
        assert before == at
        at += share
        # the last row tile is allotted a whole one's tiles, whatever it lacks of its tokens
        short = max(0, (rt + 1) * -(-rows // group) - length)
        assert abs(share / 16 - setup - tiles) <= 2 + rt / 16 + short / tile, (rt, share, tiles)
    assert at == total
