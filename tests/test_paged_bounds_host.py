"""Sizes at the ends of what the paged-cache entry points accept: calls with nothing to launch."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STORE_OF_NOTHING = """
import ctypes
import routing_dispatch_grouped_amd as rdg
A = 0x100000                            # stand-in address: nothing is launched
s = rdg.rdg_kv_step(3, 800, 16, 40000, 8192, 8192, *([A] * 8))
rc = rdg._lib.rdg_qk_norm_rope_store(A, rdg.RDG_BF16, 1024, %d, 0, 0, 128, None, None, 0.0, None, 0, 0, 0,
                                     ctypes.byref(s), None, None, 0, None)
assert rc == rdg.RDG_OK, rc
"""


@pytest.mark.parametrize("T", [1, 1023, 1024, 4096])
def test_store_without_heads_has_nothing_to_do(T):
    """No query heads and no key heads: accepted, whatever the tokens (in a process of its own, which a signal would end)."""
    done = subprocess.run([sys.executable, "-c", STORE_OF_NOTHING % T], cwd=ROOT)
    assert done.returncode == 0
