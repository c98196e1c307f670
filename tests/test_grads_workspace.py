"""Workspaces that the gradient operators keep for their callers: whose they
are and how long they live.  Tensors are on the CPU and nothing is launched.
"""

import contextlib
import os
import subprocess
import sys
import threading
import weakref

import pytest
import torch

import matrix_optimizer_step_owner_amd as mf
from matrix_optimizer_step_owner_amd import _lib, grads

CPU = torch.device("cpu")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def host(monkeypatch):
    """One stream, no GPU; `capturing` may be set."""
    state = {"capturing": False}
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(grads, "_raw_stream", lambda index: 77, raising=False)
    return state


def test_kept_from_call_to_call(host):
    a = grads._scratch(CPU, 5000, None)
    assert grads._scratch(CPU, 400, None) is a and grads._scratch(CPU, 5000, None) is a
    b = grads._scratch(CPU, 6000, None)
    assert b.numel() >= 6000 and grads._scratch(CPU, 10, None) is b


def test_host_threads_do_not_share_one(host):
    # ctypes lets another thread run between the launches of one call: two
    # threads on one stream would sort and sum in the same scratch
    got = {}

    def take(name):
        got[name] = grads._scratch(CPU, 4096, None)

    take("here")
    t = threading.Thread(target=take, args=("there",))
    t.start()
    t.join()
    assert got["here"].data_ptr() != got["there"].data_ptr()


def test_held_until_the_call_has_been_made(host, monkeypatch):
    # under capture the workspace belongs to this call alone: whoever has its
    # address has to hold it
    refs = []
    empty = torch.empty

    def watched(*args, **kwargs):
        t = empty(*args, **kwargs)
        refs.append(weakref.ref(t))
        return t

    host["capturing"] = True
    monkeypatch.setattr(torch, "empty", watched)
    held = grads._wgrad_scratch(CPU, (2, 10000, 32, 64, _lib.DTYPE_BF16), None)
    assert len(refs) == 1 and refs[0]() is not None
    del held


def test_the_steps_workspace_is_not_replaced(host, monkeypatch):
    # another thread may be in a Muon step on this stream, which goes on using
    # the address it took
    monkeypatch.setattr(mf, "_WS_CACHE", {})
    ws = mf._workspace(CPU, 77, 1000)
    grads._scratch(CPU, 100000, None)
    assert mf._workspace(CPU, 77, 1000) is ws


def test_import_without_a_gpu_backend():
    # a torch built for the CPU has none of these; the planner, the workloads
    # and the library's host functions need no GPU
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, name)\n"
            "import matrix_optimizer_step_owner_amd as mf\n"
            "from matrix_optimizer_step_owner_amd import workloads\n"
            "assert mf.CKPT_BLOCK == 128 and mf.default_scale(8, 2) == 2.0\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)


@pytest.mark.parametrize("what", [[1.0], 4096, "scratch"])
def test_arguments_that_are_not_tensors(host, what):
    with pytest.raises(TypeError, match="workspace must be a tensor"):
        grads._scratch(CPU, 256, what)
    with pytest.raises(TypeError, match="workspace must be a tensor"):
        grads._wgrad_scratch(CPU, (1, 1, 1, 1, _lib.DTYPE_BF16), what)
    with pytest.raises(TypeError, match="out must be a tensor"):
        grads._embedding_out(what, torch.bfloat16, CPU, 3, 8)
    with pytest.raises(TypeError, match="out must be a tensor"):
        grads._embedding_out(what, None, CPU, 3, 8)


def test_embedding_out():
    out = torch.zeros(3, 10)
    assert grads._embedding_out(out[:, :8], None, CPU, 3, 8) == 10
    assert grads._embedding_out(out[:, :8], torch.float32, CPU, 3, 8) == 10
    with pytest.raises(TypeError, match="expected torch.bfloat16"):
        grads._embedding_out(out[:, :8], torch.bfloat16, CPU, 3, 8)
    with pytest.raises(TypeError, match="dtype"):
        grads._embedding_out(out.double()[:, :8], None, CPU, 3, 8)
    with pytest.raises(ValueError, match="shape"):
        grads._embedding_out(out, None, CPU, 3, 8)
