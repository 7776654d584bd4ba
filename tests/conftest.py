import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


# These call the libraries with addresses that are made up or the host's, which a check has to refuse.  Where one
# does not, a kernel would be launched on them: no process that runs them may reach a GPU.
MADE_UP_ADDRESSES = ("test_abi.py", "test_serve_abi.py", "test_serve_binding.py")
_without_gpu = {}    # module: the result of its run in a process of its own


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")


def pytest_collection_finish(session):
    if not any(item.get_closest_marker("gpu") for item in session.items):
        os.environ["CUDA_VISIBLE_DEVICES"] = ""     # read when the first call initialises CUDA


def _child(target):
    return subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", target], capture_output=True,
                          text=True, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})


@pytest.hookimpl(tryfirst=True)
def pytest_pyfunc_call(pyfuncitem):
    """In a session with GPU tests, the modules above run in a child process that sees no GPU."""
    if pyfuncitem.path.name not in MADE_UP_ADDRESSES or os.environ.get("CUDA_VISIBLE_DEVICES") == "":
        return None
    module = str(pyfuncitem.path)
    if module not in _without_gpu:
        _without_gpu[module] = _child(module)
    if _without_gpu[module].returncode != 0:
        own = _child(f"{module}::{pyfuncitem.name}")
        if own.returncode != 0:
            pytest.fail(own.stdout + own.stderr, pytrace=False)
    return True


@pytest.fixture(scope="session")
def cuda_ok():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return True
