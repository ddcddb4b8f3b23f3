"""Importing the package and binding the expert-layer calls: from two threads at once, and on a
torch build without a GPU runtime."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys
import threading

import torch

from partitioned_chip_accumulation_amd import experts, hist

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_two_threads_in_their_first_call(monkeypatch):
    """The second thread calls while the first has bound one function of several."""
    halfway, resume = threading.Event(), threading.Event()

    class Library:
        bound = 0

        def __getattr__(self, name):
            if threading.current_thread() is first:
                self.bound += 1
                if self.bound == 2:
                    halfway.set()
                    assert resume.wait(60)

            def fn(*args):
                return 0
            return fn

    monkeypatch.setattr(hist, "library", lambda lib=Library(): lib)
    monkeypatch.setattr(experts, "_functions", {})
    monkeypatch.setattr(experts, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    failed = []

    def call(name):
        try:
            experts._call(name, torch.device("cuda", 0))
        except Exception as e:  # noqa: BLE001 (whatever it is, the test reports it)
            failed.append((name, e))

    first = threading.Thread(target=call, args=("experts_group",))
    first.start()
    assert halfway.wait(60)
    second = threading.Thread(target=call, args=("experts_int8_matmul",))
    second.start()
    second.join(1)  # it may end now, or wait for the first
    resume.set()
    first.join(60)
    second.join(60)
    assert not first.is_alive() and not second.is_alive()
    assert not failed
    assert set(experts._functions) == set(experts._SIGNATURES)


def test_import_without_a_gpu_runtime():
    """A torch build for the host alone lacks the GPU's entry points; the package imports there, and
    what needs no GPU works."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_getCurrent')]:\n"
            "    delattr(torch._C, name)\n"
            "import partitioned_chip_accumulation_amd as p\n"
            "from partitioned_chip_accumulation_amd import experts, hist\n"
            "assert hist.library() and p.experts is experts\n"
            "try:\n"
            "    experts.quantize_rows(torch.zeros(2, 8, dtype=torch.bfloat16))\n"
            "except ValueError:\n"
            "    print('refused')\n")
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    assert run.stdout.strip() == "refused"


def test_binding_exists_without_a_gpu():
    size = ctypes.c_uint64(0)
    assert experts._library().experts_group_workspace_size(8, 2, 4, ctypes.byref(size)) == 0
