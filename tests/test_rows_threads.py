"""The binding of the operators on logits rows when threads call it for the
first time together (no GPU: signatures only, nothing is launched)."""

import ctypes
import sys
import threading

import pytest

from speculative_decoding_verification_46_gb300 import _binding, _rows, build

NAMES = ("sv_adjust_logits", "sv_top_logits_workspace_bytes", "sv_top_logits", "sv_distill_forward", "sv_distill_backward",
         "sv_distill_loss_grad")


@pytest.fixture
def fresh(monkeypatch):
    """As in a process that has not called the library yet."""
    build.build_library()
    _rows._lib()
    monkeypatch.setattr(_binding, "_lib", None)
    monkeypatch.setattr(_rows, "_declared", type(_rows._declared)() if isinstance(_rows._declared, bool) else None)


def test_every_library_object_gets_its_signatures(fresh, monkeypatch):
    monkeypatch.setattr(_rows, "load_library", lambda: ctypes.CDLL(build.LIB_PATH))
    for _ in range(3):
        lib = _rows._lib()
        for name in NAMES:
            assert getattr(lib, name).argtypes is not None, f"{name} would be called without its signature"


def test_first_calls_of_many_threads_have_signatures(fresh):
    n, found = 8, []
    gate = threading.Barrier(n)

    def call():
        gate.wait()
        lib = _rows._lib()
        found.append([name for name in NAMES if getattr(lib, name).argtypes is None])

    old = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for _ in range(20):
            _binding._lib = None
            threads = [threading.Thread(target=call) for _ in range(n)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
    finally:
        sys.setswitchinterval(old)
    assert len(found) == 20 * n and not any(found)
