"""Tests that call the libraries with made-up addresses never run in a process that sees a GPU."""
import os
import subprocess
import sys

import pytest

from tests import conftest

SEES = """
import os
def test_sees():
    assert os.environ.get("CUDA_VISIBLE_DEVICES") == ""
def test_fails():
    assert {ok}
"""
MARKED = """
import os
import pytest
@pytest.mark.gpu
def test_marked():
    assert os.environ.get("CUDA_VISIBLE_DEVICES") is None
"""


def session(tmp_path, files):
    (tmp_path / "conftest.py").write_text(f"import sys\nsys.path.insert(0, {conftest.ROOT!r})\nfrom tests.conftest import *\n")
    for name, text in files.items():
        (tmp_path / name).write_text(text)
    env = {k: v for k, v in os.environ.items() if k != "CUDA_VISIBLE_DEVICES"}
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", str(tmp_path)], capture_output=True,
                       text=True, env=env, cwd=tmp_path)
    return r.returncode, r.stdout


@pytest.mark.parametrize("marked", [False, True])
def test_made_up_addresses_see_no_gpu(tmp_path, marked):
    files = {"test_serve_abi.py": SEES.format(ok=True), **({"test_marked.py": MARKED} if marked else {})}
    code, out = session(tmp_path, files)
    assert code == 0 and f"{3 if marked else 2} passed" in out, out


def test_a_failure_in_the_child_is_reported(tmp_path):
    code, out = session(tmp_path, {"test_serve_abi.py": SEES.format(ok=False), "test_marked.py": MARKED})
    assert code == 1 and "1 failed, 2 passed" in out and "test_fails" in out, out


def test_every_such_module_is_listed():
    here = os.path.dirname(os.path.abspath(conftest.__file__))
    address = "0x2" + 7 * "0"
    for name in os.listdir(here):
        if name.startswith("test_") and name.endswith(".py") and address in open(os.path.join(here, name)).read():
            assert name in conftest.MADE_UP_ADDRESSES, name
