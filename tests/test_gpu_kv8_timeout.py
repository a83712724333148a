"""The bounded waits of the 8-bit cache's tensor-core kernels, made to run out.

The hardware suspends a wait for longer than these kernels' phases take, so even a
limit of 1 ns is not looked at in time.  Here the two kernel files are built with
waits that poll (CSA2_POLLED_WAITS) and linked with the library's other objects; a
child process runs the calls on that library.  With the limit at 1 ns the wait
for a CTA's first tile runs out.  The kernel has to wind down (its warps leave
their loops, issued MMAs land, tensor memory is freed), report CSA2_DEV_TIMEOUT and
write nothing behind the lengths; the next call on the same workspace is right.
Nothing faults or hangs: the waits return.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

HERE = os.path.dirname(os.path.abspath(__file__))
POLLED = ("kv8_prefill.cu", "kv8_mass.cu")


def polled_library():
    from fp4_kv_cache_rope_gb300 import _build as B
    out = os.path.join(HERE, "_build")
    os.makedirs(out, exist_ok=True)
    objs, running = [], []
    for src in B.SOURCES:
        obj = os.path.join(B.BUILD, src.replace(".cu", ".o"))
        if src in POLLED:
            obj = os.path.join(out, "polled_" + src.replace(".cu", ".o"))
            running.append(subprocess.Popen(
                [B.nvcc()] + B.ARCH + B.NVCC_FLAGS + ["-DCSA2_POLLED_WAITS", "-I", os.path.join(B.ROOT, "include"),
                                                      "-c", os.path.join(B.CSRC, src), "-o", obj],
                stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL))
        objs.append(obj)
    assert [r.wait() for r in running] == [0] * len(POLLED)
    so = os.path.join(out, "libcsa2_polled.so")
    subprocess.run([B.nvcc()] + B.ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", so] + objs + ["-lcudart"],
                   check=True, capture_output=True)
    return so


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    r = subprocess.run([sys.executable, os.path.join(HERE, "kv8_timeout_child.py"), polled_library()],
                       cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.split() == ["6", "calls", "reported"]
