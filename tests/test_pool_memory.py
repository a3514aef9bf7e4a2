"""pkv_pool_* where the host has no memory left: an error code, and no exception that leaves the C entry."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# In a process of its own, whose address space may grow by 512 MB after the library is there.
CHILD = r"""
import ctypes, resource
from paged_kv_decode_block_gb300 import pkv
lib = pkv.load()
with open("/proc/self/statm") as f:
    now = int(f.read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (512 << 20), resource.RLIM_INFINITY))
pages, pool = (ctypes.c_int32 * 3)(5, 1, 7), ctypes.c_void_p(99)
for num_pages in (2 ** 31 - 1, 2 ** 28, 150 << 20):   # the marks alone are too much, or what counts the uses is
    pool.value = 99
    assert lib.pkv_pool_create(pages, 3, num_pages, ctypes.byref(pool)) == pkv.ENOMEM, num_pages
    assert not pool.value
assert lib.pkv_pool_create(pages, 3, 8, ctypes.byref(pool)) == pkv.OK and lib.pkv_pool_free_count(pool) == 3
lib.pkv_pool_destroy(pool)
print("ok")
"""


def test_a_pool_that_does_not_fit():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stderr[-2000:])
