"""What the compiler says of the cache's write: kernels that gain nothing from more CTAs an SM keep their
registers."""
import os
import re
import shutil
import subprocess

import pytest

from state_space_model_gb300 import build


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    """{kernel's mangled name: bytes of spill stores and loads} of ssd_kv.cu."""
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("needs nvcc")
    out = tmp_path_factory.mktemp("kv") / "ssd_kv.cubin"
    r = subprocess.run([build._nvcc(), *build._flags(True), "-cubin", "-o", str(out),
                        os.path.join(build.CSRC, "ssd_kv.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Function properties for (\w+)\s.*?(\d+) bytes spill stores, (\d+) bytes spill loads",
                       r.stdout + r.stderr, re.S)
    return {name: int(stores) + int(loads) for name, stores, loads in found}


def test_fp32_rows_of_one_axis_spill_nothing(report):
    kernels = {n: b for n, b in report.items() if "k_kv_appendIf" in n}
    assert len(kernels) == 12                        # 64 and 128; plain and 8 bits; one pass, two, two turned whole
    assert not any(kernels.values()), kernels
