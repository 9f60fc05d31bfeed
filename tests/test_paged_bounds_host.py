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


@pytest.mark.parametrize("T,n_req,n_q,max_q,dtype", [(4127, 32, 64, 4096, "bf16"), (8192, 64, 64, 2048, "bf16"),
                                                     (256, 256, 64, 1, "bf16"), (4096, 4096, 128, 1, "bf16"),
                                                     (100, 1, 64, 100, "bf16"), (2048, 64, 32, 1985, "bf16"),
                                                     (8192, 4, 32, 2048, "f32"), (1000, 9, 32, 500, "f32"), (64, 64, 64, 1, "f32")])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_workspace_is_bounded(T, n_req, n_q, max_q, dtype, head_dim):
    """256 MiB of the short requests' parts, and of the long ones' what 256 workgroups of 128 rows and two parts more
    a row come to, however long the contexts."""
    most = (256 << 20) + 256 + (512 + 2 * 256) * 128 * (head_dim + 2) * 4
    for max_kv in (5000, 32768, 131072, 1 << 20, (1 << 31) - 1):
        assert workspace(T, n_req, n_q, 8, head_dim, max_q, max_kv, dtype) <= most


def test_rows_that_fill_the_chip_leave_no_parts():
    for max_kv in (32768, 131072):
        assert workspace(8192, 4, 32, 8, 128, 2048, max_kv, "f32") == 0
        assert workspace(4096, 1, 64, 8, 128, 4096, max_kv, "bf16") == 0


def test_grids_that_no_launch_holds_are_refused():
    """2^32 threads and more (the runtime launches a part of them and reports nothing): refused before anything is enqueued."""
    import routing_dispatch_grouped_amd as rdg
    A = 0x100000
    c = rdg.rdg_kv_cache(4000, 16, 1, 64, A, A, A, A)

    def step(n_req, t_cap, seg_cap):
        return ctypes.byref(rdg.rdg_kv_step(n_req, 800, 16, 4000, t_cap, seg_cap, *([A] * 8)))

    def store(T, n_q, n_kv, s):
        return rdg._lib.rdg_qk_norm_rope_store(A, rdg.RDG_BF16, 4096, T, n_q, n_kv, 64, None, None, 0.0, None, 0, 0, 0, s,
                                               ctypes.byref(c), A, 4096, None)

    def attn(dtype, T, n_q, max_q, max_kv, n_req):
        return rdg._lib.rdg_paged_attention(A, dtype, n_q * 64, T, n_q, step(n_req, T, T), ctypes.byref(c), max_q, max_kv,
                                            0.1, 1, 0, A, n_q * 64, None, A, 1 << 30, None)

    assert store(1 << 27, 1, 0, step(3, 1 << 27, 0)) == rdg.RDG_EUNSUPPORTED      # 2^25 workgroups of query waves
    assert store(5, 0, 1, step(3, 1 << 26, 1 << 23)) == rdg.RDG_EUNSUPPORTED      # 2^24 of segments
    assert attn(rdg.RDG_F32, 1 << 24, 64, 1 << 24, 5000, 1) == rdg.RDG_EUNSUPPORTED   # 2^24 row tiles
    assert attn(rdg.RDG_BF16, 1 << 24, 2, 1, 5000, 2) == rdg.RDG_EUNSUPPORTED     # 2^24 tokens to join
