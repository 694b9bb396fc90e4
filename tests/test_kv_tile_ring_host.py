"""What a prefill over widened rows waits for when it gives up, on the CPU: every copy into
its shared memory that may not have landed, and no other."""
import os
import shutil
import subprocess

import pytest

from decode_megakernel_sm_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_loader_that_gives_up_drains_all_its_copies(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("compiles the account of tiles")
    program = tmp_path / "tile_ring"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", B.CSRC, os.path.join(HERE, "tile_ring.cpp"), "-o",
                    str(program)], check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True)
    assert done.returncode == 0, f"{done.stdout.strip()} findings"


def test_the_prefill_takes_its_tiles_by_that_account():
    source = open(os.path.join(B.CSRC, "kv_prefill.cuh")).read()
    assert "TileRing<NS> tiles;" in source and "tiles.take(" in source and "tiles.drain(" in source
