"""The compiled binding calls each entry point by its prototype in the library's
header, on the CPU: with one parameter more in every prototype, the binding does
not compile, and the compiler names each of them."""
import os
import re
import shutil
import subprocess
import sysconfig

import torch

from block_scaled_precision_02_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
QUANT = ("i8_rowwise", "f8_pertoken", "f8_block", "mx")
ENTRIES = (["qgemm_moe_sort_workspace", "qgemm_moe_sort", "qgemm_moe_gather", "qgemm_moe_combine", "qgemm_moe_combine_grad"] +
           [f"qgemm_{o}_quant_{k}" for o in ("swiglu", "postnorm") for k in QUANT] +
           [f"qgemm_{k}_grouped" for k in ("i8_rowwise", "f8_pertoken", "f8_blockscale", "mx")])


def test_a_changed_prototype_does_not_compile(tmp_path):
    csrc = tmp_path / "package" / "csrc" / "binding"
    csrc.mkdir(parents=True)
    (tmp_path / "include").mkdir()
    shutil.copy(build.FAST_SRC, csrc / "fast.cpp")
    header = open(os.path.join(ROOT, "include", "qgemm.h")).read()
    for name in ENTRIES:
        header, n = re.subn(rf"\b{name}\(([^)]*)\);", rf"{name}(\1, struct more_{name} *more);", header)
        assert n == 1, name
    (tmp_path / "include" / "qgemm.h").write_text(
        "".join(f"struct more_{name};\n" for name in ENTRIES) + header)
    base = os.path.dirname(torch.__file__)
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"]]
    r = subprocess.run([os.environ.get("CXX", "g++"), "-fsyntax-only", "-std=c++17", "-fmax-errors=0"] +
                       [f"-isystem{d}" for d in include] + [str(csrc / "fast.cpp")], capture_output=True, text=True)
    assert r.returncode != 0
    missing = [name for name in ENTRIES if not re.search(rf"\bmore_{name}\b", r.stderr)]
    assert not missing, missing
