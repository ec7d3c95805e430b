"""The first call of the process: a library that fails to load, and two threads at once.  No GPU."""
import subprocess
import sys
import threading

import pytest
import torch

from convolution_implicit_gemm_amd import FusedConvError
from convolution_implicit_gemm_amd import transformer as T


@pytest.fixture
def unused(monkeypatch):
    """The module as it is before its first call."""
    monkeypatch.setattr(T, "torch", None)
    monkeypatch.setattr(T, "_DTYPES", {})
    monkeypatch.setattr(T, "_current_handle", None)
    monkeypatch.setattr(T, "_calls", {})


def test_a_failing_load_is_reported_every_time(unused, monkeypatch):
    def fail():
        raise RuntimeError("no library here")

    monkeypatch.setattr(T, "_load", fail)
    x = torch.zeros(4, 16)
    for _ in range(3):
        with pytest.raises(RuntimeError, match="no library here"):
            T.layer_norm(x)
    monkeypatch.undo()
    with pytest.raises(FusedConvError, match="device tensor"):  # and the next call can succeed
        T.layer_norm(x)


def test_two_threads(unused, monkeypatch):
    """The second thread's first call comes while the first one's is still loading."""
    loading, go_on = threading.Event(), threading.Event()
    load = T._load

    def slow():
        loading.set()
        assert go_on.wait(30)
        return load()

    monkeypatch.setattr(T, "_load", slow)
    seen = []

    def call():
        try:
            T.layer_norm(torch.zeros(4, 16))
        except Exception as e:  # noqa: BLE001
            seen.append(e)

    threads = [threading.Thread(target=call) for _ in range(2)]
    threads[0].start()
    assert loading.wait(30)
    threads[1].start()
    threads[1].join(0.5)
    go_on.set()
    for t in threads:
        t.join(30)
    assert len(seen) == 2
    for e in seen:
        assert isinstance(e, FusedConvError) and "device tensor" in str(e), repr(e)


def test_import_needs_no_torch():
    code = "import sys, convolution_implicit_gemm_amd; sys.exit('torch' in sys.modules)"
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0
