"""What calls from several threads share on the host, under a thread checker."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "trellis_coded_quantized_amd", "csrc")


def test_lds_limits_are_raised_from_several_threads(tmp_path):
    exe = str(tmp_path / "lds_limit")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-I", os.path.join(HERE, "host"), "-I", CSRC,
                    os.path.join(HERE, "host", "lds_limit.cpp"), "-o", exe, "-lpthread"], check=True)
    run = subprocess.run([exe], capture_output=True, text=True)
    if "unexpected memory mapping" in run.stderr:
        pytest.skip("the thread checker cannot map its memory on this machine")
    assert run.returncode == 0, run.stderr[-2000:]
