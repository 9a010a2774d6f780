"""The 8-bit float product's map from workgroups to tiles (lds_tiles.hpp), compiled for the host:
every tile is one workgroup's, also in a grid that is larger than the product's own, which the
smaller one of two gradients gets where both share a launch. A second workgroup would compute a
tile again and store to the same addresses at the same time."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_every_tile_is_one_workgroups(tmp_path):
    if not os.path.exists(HIPCC) and not shutil.which("hipcc"):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "tile_map")
    subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-std=c++17", "-I",
                    os.path.join(ROOT, "bitwise_consistent_linear_amd", "csrc"), "-o", exe,
                    os.path.join(ROOT, "tests", "tile_map.cpp")], check=True, capture_output=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(lines) == 8 * 6 * 5 + 1
    wrong = [line for line in lines if not line.endswith("least=1 most=1 outside=0")]
    assert not wrong, (len(wrong), wrong[:5], lines[-1])
