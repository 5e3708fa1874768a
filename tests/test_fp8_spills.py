"""What the kernels of fp8_pack.cu spill, as the compiler reports it.

The launch bounds of fp8_pack_rows are chosen by type: a bound that suits bf16 made fp32 rows with
silu spill 580 bytes a thread, more than a thread reads of x, for twice the time.
"""
import os
import re
import subprocess

from int4_quantized_b200 import _build

CSRC = os.path.join(os.path.dirname(__file__), "..", "int4_quantized_b200", "csrc")


def test_pack_kernels_spill_little(tmp_path):
    flags = [f for f in _build.NVCC_FLAGS if f != "-shared"]
    out = subprocess.run([_build.nvcc(), *flags, "-Xptxas", "-v", "-c", "-o", str(tmp_path / "o.o"), os.path.join(CSRC, "fp8_pack.cu")],
                         capture_output=True, text=True, check=True).stderr
    kernels = re.findall(r"entry function '([^']+)'.*?(\d+) bytes spill stores, (\d+) bytes spill loads", out, re.S)
    assert len(kernels) == 30
    for name, stores, loads in kernels:
        assert int(stores) <= 96 and int(loads) <= 96, (name, stores, loads)
