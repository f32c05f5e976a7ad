"""The attention binding where torch has no 4-bit element type: all other pools are served."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
if hasattr(torch, "float4_e2m1fn_x2"):
    del torch.float4_e2m1fn_x2
from state_space_model_gb300 import attn
pool = torch.zeros(1, 1, 16, 64)
for call in (lambda: attn.kv_read(pool, pool, None, None, 1, dtype=torch.float16),
             lambda: attn.kv_read(pool.bfloat16(), pool.bfloat16(), None, None, 1, dtype=torch.float32)):
    try:
        call()
    except ValueError as e:
        print(e)
"""


def test_module_without_the_type():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.splitlines() == ["rows of torch.float32 pools cannot be read as torch.float16",
                                     "rows of torch.bfloat16 pools cannot be read as torch.float32"]


PROGRAM = """
#include "scalar_types.h"
enum class Old { Float, Byte };
enum class New { Float, Byte, Float4_e2m1fn_x2 };
static_assert(!FourBits<Old>::is(Old::Float) && !FourBits<Old>::is(Old::Byte));
static_assert(FourBits<New>::is(New::Float4_e2m1fn_x2) && !FourBits<New>::is(New::Byte));
int main() { return 0; }
"""


def test_binding_without_the_type(tmp_path):
    """The binding names the type through one header only, which compiles with and without it."""
    if not shutil.which("g++"):
        pytest.skip("needs g++")
    binding = os.path.join(ROOT, "state_space_model_gb300", "binding")
    with open(os.path.join(binding, "attn_ext.cpp")) as f:
        assert "Float4" not in f.read()
    src = tmp_path / "types.cpp"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-I", binding, str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
