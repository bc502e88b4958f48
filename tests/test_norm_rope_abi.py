"""Refusals of the query/key norm's C entries on the CPU (no pointer here is ever
dereferenced): outputs that lie on weights, tables, positions, the workspace or each
other would be read after they are written."""
import ctypes

import pytest

from linear_attention_recurrence_fwd_amd import binding as B

INVALID = 1
# sizes in bytes: B T = 10 tokens, heads of 64 channels, a table of 4096 x 32
Q, K, W, ROPE, POS = 10 * 4 * 64 * 2, 10 * 2 * 64 * 2, 64 * 4, 4096 * 32 * 4, 10 * 4


def dims():
    return B.NormDims(2, 5, 4, 2, 64, 32, 4096, 0, 0, B.GDN_BF16, 0, 1e-6, 0.0)


def places(n):
    return [ctypes.c_void_p((1 << 30) + i * (1 << 20)) for i in range(n)]


def shifts(out, other):
    """All of the other, its last 16 bytes, and its first 16."""
    return (0, max(0, (other - 4) // 16 * 16), -(out - 16))


@pytest.mark.parametrize("out,n", [(6, Q), (7, K)])
@pytest.mark.parametrize("other,m", [(2, W), (3, W), (4, ROPE), (5, POS)])
def test_forward_outputs_off_weights_table_and_positions(out, n, other, m):
    for shift in shifts(n, m):
        a = places(8)  # q k wq wk rope pos oq ok
        a[out] = ctypes.c_void_p(a[other].value + shift)
        assert B.lib().gdn_norm_rope_fwd(ctypes.byref(dims()), *a, None) == INVALID, shift


@pytest.mark.parametrize("out,n", [(8, Q), (9, K)])
@pytest.mark.parametrize("other,m", [(2, W), (3, W), (4, ROPE), (5, POS), (10, W), (11, W)])
def test_backward_rows_off_weights_table_positions_and_weight_gradients(out, n, other, m):
    for shift in shifts(n, m):
        a = places(12)  # q k wq wk rope pos dyq dyk dq dk dwq dwk
        a[out] = ctypes.c_void_p(a[other].value + shift)
        ws = ctypes.c_void_p(1 << 28)
        assert B.lib().gdn_norm_rope_bwd(ctypes.byref(dims()), *a, ws, 1 << 20, None) == INVALID, shift


def test_weight_gradients_off_each_other_and_the_workspace():
    need = ctypes.c_size_t(0)
    assert B.lib().gdn_norm_rope_bwd_workspace_bytes(ctypes.byref(dims()), ctypes.byref(need)) == 0 and need.value >= 32
    for shift in shifts(W, W):
        a = places(12)
        a[10] = ctypes.c_void_p(a[11].value + shift)
        assert B.lib().gdn_norm_rope_bwd(ctypes.byref(dims()), *a, ctypes.c_void_p(1 << 28), 1 << 20, None) == INVALID, shift
    for i in (10, 11):
        for shift in (0, need.value - 16, -(W - 16)):
            a = places(12)
            a[i] = ctypes.c_void_p((1 << 28) + shift)
            assert B.lib().gdn_norm_rope_bwd(ctypes.byref(dims()), *a, ctypes.c_void_p(1 << 28), 1 << 20, None) == INVALID, shift
    for i in (2, 3, 4, 5):  # the workspace on what is read
        a = places(12)
        assert B.lib().gdn_norm_rope_bwd(ctypes.byref(dims()), *a, a[i], 1 << 20, None) == INVALID


def test_nothing_overlaps_no_bytes():
    """Without tokens there is nothing to write, wherever the outputs point (and no launch)."""
    d = B.NormDims(2, 0, 4, 2, 64, 32, 4096, 0, 0, B.GDN_BF16, 0, 1e-6, 0.0)
    for out in (6, 7):
        for other in (2, 3, 4):
            a = places(8)
            a[out] = ctypes.c_void_p(a[other].value + 16)
            assert B.lib().gdn_norm_rope_fwd(ctypes.byref(d), *a, None) == 0, (out, other)
