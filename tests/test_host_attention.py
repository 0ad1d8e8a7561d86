"""Device code of the attention kernels that exchanges nothing between lanes,
compiled for the CPU and run a lane at a time (tests/host/)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "trellis_coded_quantized_amd", "csrc")
CLANG = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "clang++")


def compiled(name, folder):
    exe = os.path.join(str(folder), name)
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O1", "-w", "-I", os.path.join(HERE, "host"), "-I", CSRC,
                    os.path.join(HERE, "host", name + ".cpp"), "-o", exe], check=True)
    return exe


@pytest.fixture(scope="module")
def nonfinite_values(tmp_path_factory):
    return compiled("nonfinite_values", tmp_path_factory.mktemp("host"))


# tiles of 32 keys (few rows) and of 64 (many rows); tables that end with a tile and inside one
@pytest.mark.parametrize("keys,page_log2,width", [
    (32, 4, 1), (32, 4, 2), (32, 4, 3), (32, 5, 1), (64, 4, 1), (64, 4, 4), (64, 4, 5), (64, 4, 6), (64, 4, 7),
    (64, 5, 2), (64, 5, 3), (64, 6, 1), (64, 8, 1)])
def test_infinities_are_put_back_without_reading_past_the_table(nonfinite_values, keys, page_log2, width):
    assert subprocess.run([nonfinite_values, str(keys), str(page_log2), str(width)]).returncode == 0
