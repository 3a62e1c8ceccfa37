"""The binding's stream argument, on CPU: a given stream needs no torch, and the current stream's address is taken the
short way as soon as CUDA is initialised, whatever the first call was."""
import os
import subprocess
import sys
import types

import pytest

k3 = pytest.importorskip("lossless_bf16_weight_k3huf_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_given_stream_needs_no_torch():
    code = ("import sys; sys.modules['torch'] = None\n"
            "import lossless_bf16_weight_k3huf_gb300 as k3\n"
            "class S: cuda_stream = 77\n"
            "assert k3._stream(5) == 5 and k3._stream(0) == 0 and k3._stream(S()) == 77\n"
            "try: k3._stream(None)\n"
            "except ImportError: pass\n"
            "else: raise AssertionError('the current stream is torch\\'s')\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)


def test_calls_before_cuda_is_initialised_do_not_decide(monkeypatch):
    torch = types.ModuleType("torch")
    up, slow = [False], []
    torch.cuda = types.SimpleNamespace(is_initialized=lambda: up[0], current_stream=lambda: slow.append(1) or types.SimpleNamespace(cuda_stream=11))
    torch._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda device: 100 + device, _cuda_getDevice=lambda: 2)
    monkeypatch.setitem(sys.modules, "torch", torch)
    monkeypatch.setattr(k3, "_raw_stream", None)
    assert k3._stream(5) == 5
    assert k3._stream(None) == 11 and len(slow) == 1     # (CUDA not initialised: torch does so)
    up[0] = True
    assert k3._stream(None) == 102 and len(slow) == 1
    assert k3._stream(7) == 7
