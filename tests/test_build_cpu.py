"""What build() makes: the binding module finds the library beside it wherever the package
lies."""
import os
import shutil
import subprocess
import sys

import pytest

import exact_io_aware_27_gb300 as fa
from exact_io_aware_27_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()


def test_a_copied_package_uses_its_own_library(tmp_path):
    name = os.path.basename(_build.PKG_DIR)
    copy = tmp_path / name
    copy.mkdir()
    for f in os.listdir(_build.PKG_DIR):
        if f.endswith((".py", ".so")):
            shutil.copy2(os.path.join(_build.PKG_DIR, f), copy)
    code = (f"import sys; sys.path.insert(0, {str(tmp_path)!r})\n"
            f"from {name} import packed\n"
            "packed._binding()\n"
            "print(*{l.split()[-1] for l in open('/proc/self/maps') if 'libfa_gb300' in l"
            " or '_fa_binding' in l}, sep='\\n')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=tmp_path, timeout=300)
    assert r.returncode == 0, r.stderr
    assert sorted(r.stdout.split()) == sorted(str(copy / os.path.basename(f))
                                              for f in (_build.BINDING, _build.LIBRARY))


def test_the_binding_of_another_torch_is_not_used():
    """The module is built against one torch and one Python; with another torch it is not
    loaded, and build() has work to do."""
    name = os.path.basename(_build.PKG_DIR)
    code = ("import torch\n"
            "torch.__version__ = '0.0.1'\n"
            f"from {name} import _build, packed\n"
            "assert not _build.up_to_date()\n"
            "try:\n"
            "    packed._binding()\n"
            "except RuntimeError as e:\n"
            "    assert 'is not built' in str(e), e\n"
            "    print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=_build.ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["refused"], r.stdout + r.stderr
    assert _build.up_to_date()
