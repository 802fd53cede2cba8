"""The binding's host helper belongs to the model-step operators alone: without
it the collectives import and build as ever, and the operators say what is
missing.  Needs no GPU."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "collective_communication_primitives_amd"


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)


@pytest.mark.parametrize("how", ["absent", "for another torch"])
def test_the_collectives_do_without_the_helper(how):
    block = f"sys.modules['{PACKAGE}._marshal'] = None\n" if how == "absent" else (
        "import types\nm = types.ModuleType('m')\nm.torch_version = 'another'\nm.buffers = m.counts = None\n"
        f"sys.modules['{PACKAGE}._marshal'] = m\n")
    run = python("import sys\n" + block + f"""
import torch, {PACKAGE} as dt
assert dt.version() and dt.dt_layer_norm_workspace([4], 8) > 0
torch.cuda.current_device = lambda: -1
x = [torch.zeros(4, 8)]
try:
    dt.dt_layer_norm(x, [torch.ones(8)], None, [torch.zeros(4, 8)])
except ImportError as e:
    assert 'build.py' in str(e), e
    print('said')
""")
    assert run.returncode == 0 and run.stdout.strip() == "said", run.stdout + run.stderr


def test_the_library_is_built_where_the_helper_cannot_be(monkeypatch, tmp_path):
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, PACKAGE, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    for name, to in (("LIBRARY", "lib.so"), ("MARSHAL", "helper.so"), ("BUILD_DIR", "objects")):
        monkeypatch.setattr(build, name, str(tmp_path / to))

    def run(cmd, **_):  # no compiler: hipcc's outputs are empty files, g++ finds no headers
        failed = "++" in os.path.basename(cmd[0])
        if not failed:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(failed), "", "no Python.h" if failed else "")

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no Python.h"):
        build.build()
    assert os.path.exists(build.LIBRARY) and not os.path.exists(build.MARSHAL)


def test_the_helper_is_tagged_for_this_python():
    from collective_communication_primitives_amd import _marshal
    assert "cpython-%d%d" % sys.version_info[:2] in os.path.basename(_marshal.__file__)
