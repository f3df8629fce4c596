"""A C entry that finds no host memory returns an error: no exception leaves the
library (CPU; a child process with a bounded address space)."""
import subprocess
import sys

import fp8_block_scaled_10_b200 as fp8bs

CHILD = r"""
import ctypes, resource
lib = ctypes.CDLL(%r)
n = 1 << 20
grads = (ctypes.c_uint64 * n)(*range(1 << 30, (1 << 30) + 64 * n, 64))
sizes = (ctypes.c_int64 * n)(*[16] * n)
types = (ctypes.c_int * n)(*[1] * n)
bound = ctypes.c_double(1.0)
lib.fp8bs_last_error_message.restype = ctypes.c_char_p
def call(count):
    return lib.fp8bs_clip_grads(grads, grads, sizes, types, types, ctypes.c_int64(count), ctypes.byref(bound),
                                ctypes.c_void_p(4096), None, ctypes.c_size_t(0), None)
used = int(next(l for l in open("/proc/self/status") if l.startswith("VmSize")).split()[1]) * 1024
resource.setrlimit(resource.RLIMIT_AS, (used + (4 << 20), resource.RLIM_INFINITY))
first = call(n)                        # 24 MB of ranges: refused
message = lib.fp8bs_last_error_message().decode()
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
print(first, "|", message)
"""


def test_clip_without_host_memory_is_an_error():
    fp8bs.lib()
    out = subprocess.run([sys.executable, "-c", CHILD % fp8bs.LIB_PATH], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, (out.returncode, out.stderr[-500:])
    status, message = out.stdout.split("|", 1)
    assert int(status) == fp8bs.ERR_WORKSPACE and "host memory" in message
