"""The order of the LDS stages in the matrix products' kernels of the built library
(no GPU), as the loss' kernels are followed: no stage is loaded again over reads
that may still be on their way."""
import os
import shutil
import subprocess

import pytest

from collective_communication_primitives_amd import _lib
from test_loss_stages import OBJDUMP, functions, stale_reads


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    where = tmp_path_factory.mktemp("code")
    shutil.copy(_lib.LIBRARY, where / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=where, check=True, capture_output=True)
    found = {}
    for name in sorted(os.listdir(where)):
        if "gfx950" in name:
            with open(where / name, "rb") as f:
                if b"k_linear_dweight" not in f.read():
                    continue
            out = subprocess.run([OBJDUMP, "-d", name], cwd=where, check=True, capture_output=True, text=True).stdout
            found.update({k: v for k, v in functions(out).items() if "k_linear" in k and "Shape" in k})
    return found


def test_no_stage_is_loaded_over_outstanding_reads(kernels):
    for form in ("k_linearI", "k_linear_dxI", "k_linear_dweightI"):
        assert sum(form in k for k in kernels) >= 4, form
    bad = {k: ["%x" % a for a in at] for k, v in kernels.items() if (at := stale_reads(v))}
    assert bad == {}
