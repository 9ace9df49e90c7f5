"""The binding's host-side calls are built against one PyTorch's and one Python's binary interface: they
are found by that, and without them, or with a file that does not load, every call goes the longer way
(no GPU needed)."""

import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import build as B
from moe_grouped_matrix_gb300 import moe


@pytest.fixture(scope="module", autouse=True)
def library():
    B.build()
    G.load_library()


@pytest.fixture
def unbound(monkeypatch):
    monkeypatch.setattr(moe, "_calls", None)


def test_the_file_is_this_pytorchs_and_this_pythons(monkeypatch):
    path = B.host_calls_path()
    assert os.path.exists(path)
    assert torch.__version__ in path and path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "9.9.9+cu990")
    assert B.host_calls_path() != path and B._stale(B.host_calls_path(), [B.HOST_CALLS])


def refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA tensor"):
        G.route(torch.zeros((4, 8)), 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        G.quantize_fp4(torch.zeros((4, 64)))


def test_the_built_file_binds(unbound, recwarn):
    refuses_host_tensors()
    assert not isinstance(moe._calls, moe._NoCalls) and not recwarn


def test_another_pytorch_does_not_load_it(unbound, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "9.9.9+cu990")
    with pytest.warns(RuntimeWarning, match="longer way"):
        refuses_host_tensors()
    assert isinstance(moe._calls, moe._NoCalls)


def test_a_file_that_does_not_load(unbound, monkeypatch, tmp_path):
    bad = tmp_path / "_host_calls.so"
    bad.write_bytes(b"no library")
    monkeypatch.setattr(B, "host_calls_path", lambda: str(bad))
    with pytest.warns(RuntimeWarning, match="longer way"):
        refuses_host_tensors()


WITHOUT_CUDA = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
torch.version.cuda = None
import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import build as B
B._host_calls_command = None
B.HERE = B.BUILD_DIR  # where no host-side calls are
B.build()
for call in (lambda: G.route(torch.zeros((4, 8)), 2), lambda: G.gmm(*[torch.zeros(2, 2, 2)] * 3)):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e)
    else:
        raise AssertionError
"""


def test_a_pytorch_without_cuda_imports_and_builds():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-W", "ignore", "-c", WITHOUT_CUDA], cwd=root, capture_output=True, text=True)
    assert got.returncode == 0, got.stderr[-2000:]
