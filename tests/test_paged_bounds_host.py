"""Sizes at the ends of what the paged-cache entry points accept: calls with nothing to launch."""
import ctypes
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


def workspace(T, n_req, n_q, n_kv, head_dim, max_q, max_kv, dtype):
    import routing_dispatch_grouped_amd as rdg
    A = 0x100000
    c = rdg.rdg_kv_cache(40, 16, n_kv, head_dim, A, A, A, A)
    return rdg._lib.rdg_paged_attention_workspace_bytes(ctypes.byref(c), T, n_req, n_q, max_q, max_kv,
                                                        rdg.RDG_BF16 if dtype == "bf16" else rdg.RDG_F32)


@pytest.mark.parametrize("max_kv", [3000, 16384, 131072])
@pytest.mark.parametrize("T", [2100, 4127, 20000])
def test_workspace_of_a_mixed_batch_is_that_of_its_short_requests(T, max_kv):
    """A long prefill chunk beside 31 decode rows: its tokens, whose keys are not split, take no room for the decode rows' parts."""
    short = 8                                # queries of 8 heads a key head that a 64-row workgroup takes
    alone = workspace(32 * short, 32, 64, 8, 128, short, max_kv, "bf16")
    assert 0 < workspace(T, 32, 64, 8, 128, T - 31, max_kv, "bf16") == alone
