"""BlockAllocator calls that give blocks back need no memory of their own: a
process that has none left must get through them."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_220_gb300 import build

CODE = """
import resource, sys
sys.path.insert(0, %r)
import paged_kv_cache_220_gb300 as pkv
n = 1 << 21
a = pkv.BlockAllocator(n, 1, seed=1)
s = a.new_seq()
a.append(s, n)
if sys.argv[1] == "loaded":
    a = pkv.BlockAllocator.load(a.save())
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + (1 << 20), resource.RLIM_INFINITY))
a.truncate(s, 5)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
print(a.seq_len(s), a.stats()["free_blocks"] == n - 5)
"""


@pytest.mark.parametrize("how", ["made", "loaded"])
def test_truncate_without_memory(how):
    build.build()
    # large pieces come from the system and go back to it at once
    env = dict(os.environ, MALLOC_MMAP_THRESHOLD_="65536")
    r = subprocess.run([sys.executable, "-c", CODE % os.path.dirname(build.HERE), how],
                       capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.split() == ["5", "True"]
