"""The package on a torch that lacks a type which only the 8-bit cache needs."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
torch.__dict__.pop("{name}", None)
import trellis_coded_quantized_amd as tq
tq.load_library()
assert callable(tq.matvec_axis1) and callable(tq.kv_cache)
k, v = tq.kv_cache(1, 2, 1, 64, 16, device="cpu")
for call in (lambda: tq.kv8_cache(1, 2, 1, 64, 16, device="cpu"),
             lambda: tq.cache_fork_kv8(k, v, None, None, None, None, None, None, None),
             lambda: tq.tree_attention_kv8(k, k, v, None, None, None, None, None, None, 1),
             lambda: tq.qk_norm_rope_kv8(k, k, v, None, None, None, None, None, k, v, None, None)):
    try:
        call()
    except TypeError as e:
        assert "{name}" in str(e), e
    else:
        raise AssertionError("not refused")
"""


@pytest.mark.parametrize("name", ["float8_e8m0fnu", "float8_e4m3fn"])
def test_a_torch_without_the_8_bit_types(name):
    done = subprocess.run([sys.executable, "-c", CODE.format(name=name)], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
