"""The size query of the attention over pages and the call agree, on the CPU: what the query
asks for with the max_q that the call takes is what the call needs, no more and no less
(the launches are not reached: the call is made with one byte less than is needed, or is
refused for a misplaced output behind the workspace's check)."""
import ctypes

import pytest

from linear_attention_recurrence_fwd_amd import binding as B
from test_paged_abi import INVALID, OK, WORKSPACE, places, pool_dims


def query(d, prefix, max_q, max_len):
    need = ctypes.c_size_t(0)
    assert B.lib().gdn_prefix_attention_workspace_bytes(ctypes.byref(d), prefix, max_q, max_len, ctypes.byref(need)) == OK
    return need.value


def attend(d, prefix, max_q, max_len, ws, uniform):
    """The call with its output on its queries, which is looked at behind the workspace's size."""
    p = places(10)  # q k v table lens prefix_pages cu o lse ws
    return B.lib().gdn_prefix_attention(ctypes.byref(d), *p[:6], prefix, None if uniform else p[6], max_q, max_len, 1.0, p[0],
                                        p[8], p[9], ws, None)


@pytest.mark.parametrize("dtype", [B.GDN_BF16, B.GDN_F32])
@pytest.mark.parametrize("N,S", [(64, 64), (64, 8), (64, 1), (1000, 10), (4096, 16)])
@pytest.mark.parametrize("prefix,max_len", [(0, 96), (100, 96), (32768, 4000), (0, 100000), (70001, 0)])
def test_without_cu_by_n_over_s(N, S, prefix, max_len, dtype):
    """With N / S the query's size is the call's, whatever max_q the call is given."""
    d = pool_dims(N=N, S=S, width=8000, dtype=dtype)
    need = query(d, prefix, N // S, max_len)
    for max_q in (1, N // S, N // 2, N, 0, -1, N + 1):
        assert attend(d, prefix, max_q, max_len, need, True) == INVALID
        if need:
            assert attend(d, prefix, max_q, max_len, need - 1, True) == WORKSPACE


@pytest.mark.parametrize("max_q", [1, 5, 33, 64])
@pytest.mark.parametrize("prefix,max_len", [(0, 96), (32768, 4000), (0, 100000)])
def test_with_cu_by_max_q(max_q, prefix, max_len):
    d = pool_dims(N=64, S=8, width=8000)
    need = query(d, prefix, max_q, max_len)
    assert attend(d, prefix, max_q, max_len, need, False) == INVALID
    if need:
        assert attend(d, prefix, max_q, max_len, need - 1, False) == WORKSPACE
