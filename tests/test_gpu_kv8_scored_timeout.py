"""The bounded waits of the many-row attention with changed scores, made to run out, as
test_gpu_kv8_timeout.py does it for the other tensor-core kernels: a build whose waits
poll, a limit of 1 ns, the status, and a right next call.  Nothing faults or hangs."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import test_gpu_kv8_timeout as base  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(monkeypatch):
    monkeypatch.setattr(base, "POLLED", ("kv8_scored_prefill.cu",))
    r = subprocess.run([sys.executable, os.path.join(HERE, "kv8_scored_timeout_child.py"),
                        base.polled_library()], cwd=os.path.dirname(HERE), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.split() == ["16", "calls", "reported"]
