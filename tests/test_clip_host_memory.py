"""Clipping a list too long for the host's memory says so (and not that its tensors overlap)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import ctypes as C, resource, sys
import numpy as np
import fine_grained_blockwise_amd as fgb
L = fgb.lib()
n = 6 * 10 ** 6  # 2 n entries of 24 bytes and more: 288 MB at least
at = (0x100000 + 64 * np.arange(n)).astype(np.uint64)
out = at + (1 << 40)
length, kind = np.full(n, 8, np.int64), np.zeros(n, np.int32)
p = lambda a: C.c_void_p(a.ctypes.data)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
if sys.argv[1] == "short":
    resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 26), resource.RLIM_INFINITY))
# (norm is missing: nothing is enqueued)
rc = L.grad_clip(p(at), p(out), p(length), p(kind), p(kind), n, 1.0, 1.0, C.c_void_p(0x1000), None, None, 0, None)
print("rc", rc, L.fgb_last_error().decode())
"""


def run(how):
    r = subprocess.run([sys.executable, "-c", CODE, how], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_no_host_memory():
    out = run("short")
    assert "rc 5" in out and "host memory" in out
    out = run("enough")
    assert "rc 1" in out and "norm null" in out
