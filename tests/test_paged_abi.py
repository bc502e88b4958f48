"""Refusals of the rotation with several axes, of appending to a paged cache and of the
attention over it, on the CPU: C entries with places that are never read, and the
binding's checks."""
import ctypes

import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def places(n):
    return [ctypes.c_void_p((1 << 40) + i * (1 << 36)) for i in range(n)]


def pool_dims(**kw):
    """70 tokens of 4 sequences, 8 over 2 heads of 64, 100 pages of 16, head by head."""
    d = dict(N=70, S=4, Hq=8, Hk=2, D=64, pages=100, page=16, width=6, page_stride=2 * 16 * 64, head_stride=16 * 64,
             token_stride=64, dtype=B.GDN_BF16)
    d.update(kw)
    return B.PagedDims(*[d[n] for n, _ in B.PagedDims._fields_])


def turn(**kw):
    t = dict(P=50, R=32, q_stride=0, k_stride=0, v_stride=0, first=0, A=3, interleaved=0, eps=1e-6, w_offset=0.0)
    t.update(kw)
    return B.Turn(*[t[n] for n, _ in B.Turn._fields_])


# ------------------------------------------------------------ rotation with several axes

def axes_dims(**kw):
    d = dict(B=2, T=5, Hq=4, Hk=2, D=64, R=32, P=50, q_stride=0, k_stride=0, dtype=B.GDN_BF16, interleaved=0, eps=1e-6,
             w_offset=0.0)
    d.update(kw)
    return B.NormDims(*[d[n] for n, _ in B.NormDims._fields_])


def axes_fwd(d, A=3, **at):
    p = places(9)  # q k wq wk rope axis pos oq ok
    for i, x in at.items():
        p[int(i[1:])] = x
    return B.lib().gdn_norm_rope_axes_fwd(ctypes.byref(d), A, *p, None)


def axes_bwd(d, A=3, need=1 << 30, **at):
    p = places(14)  # q k wq wk rope axis pos dyq dyk dq dk dwq dwk ws
    for i, x in at.items():
        p[int(i[1:])] = x
    return B.lib().gdn_norm_rope_axes_bwd(ctypes.byref(d), A, *p, need, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(R=80), INVALID), (dict(eps=-1.0), INVALID), (dict(q_stride=8), INVALID),
    (dict(D=12), UNSUPPORTED), (dict(D=520), UNSUPPORTED), (dict(R=24), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED)])
def test_axes_dims(kw, code):
    assert axes_fwd(axes_dims(**kw)) == code and axes_bwd(axes_dims(**kw)) == code


def test_axes_arguments():
    d = axes_dims()
    for A, code in ((0, INVALID), (-1, INVALID), (5, UNSUPPORTED)):
        assert axes_fwd(d, A) == code and axes_bwd(d, A) == code
    one = ctypes.c_void_p((1 << 40) + 8)
    for i in (0, 1, 2, 3, 4, 7, 8):  # absent (of the weights one alone), off 16 bytes
        assert axes_fwd(d, **{"_%d" % i: None}) == INVALID, i
        assert axes_fwd(d, **{"_%d" % i: one}) == INVALID, i
    for i in (0, 1, 2, 3, 4, 7, 8, 9, 10, 11, 12):
        assert axes_bwd(d, **{"_%d" % i: None}) == INVALID, i
    assert axes_bwd(d, _13=None) == WORKSPACE and axes_bwd(d, need=16) == WORKSPACE
    # without the norm: no weights, no q and k, no workspace
    bare = dict(_0=None, _1=None, _2=None, _3=None, _11=None, _12=None, _13=None)
    for i in (4, 7, 8, 9, 10):
        assert axes_bwd(d, need=0, **{**bare, "_%d" % i: None}) == INVALID, i


def test_axes_overlaps():
    d = axes_dims()
    p = places(14)
    q, k = 10 * 4 * 64 * 2, 10 * 2 * 64 * 2
    size = {0: q, 1: k, 2: 256, 3: 256, 4: 50 * 32 * 4, 5: 16, 6: 3 * 10 * 4}

    def at(i, shift):
        return ctypes.c_void_p(p[i].value + shift)

    for out, n in ((7, q), (8, k)):
        for other, m in size.items():
            for shift in (0, (m - 1) // 16 * 16, 16 - n):
                assert axes_fwd(d, **{"_%d" % out: at(other, shift)}) == INVALID, (out, other, shift)
    assert axes_fwd(d, _7=at(8, k - 16)) == INVALID
    for out, n in ((9, q), (10, k)):
        for other, m in {**size, 7: q, 8: k, 11: 256, 12: 256}.items():
            for shift in (0, (m - 1) // 16 * 16, 16 - n):
                assert axes_bwd(d, **{"_%d" % out: at(other, shift)}) == INVALID, (out, other, shift)


# ----------------------------------------------------------------------------- appending

def append(d, t=None, **at):
    p = places(14)  # q k v wq wk rope axis pos table past cu oq k_pages v_pages
    for i, x in at.items():
        p[int(i[1:])] = x
    return B.lib().gdn_paged_append(ctypes.byref(d), ctypes.byref(t or turn()), *p, None)


POOL = [(dict(N=-1), INVALID), (dict(S=0), INVALID), (dict(Hk=0), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
        (dict(width=0), INVALID), (dict(D=0), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(D=12), UNSUPPORTED),
        (dict(D=264), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=8192), UNSUPPORTED),
        (dict(token_stride=56), INVALID), (dict(token_stride=68), INVALID), (dict(head_stride=512), INVALID),
        (dict(page_stride=1024), INVALID), (dict(page_stride=-2048), INVALID), (dict(head_stride=0), INVALID),
        (dict(page_stride=1 << 41), INVALID), (dict(page_stride=1 << 40, pages=1 << 30), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", POOL)
def test_pool_dims(kw, code):
    d = pool_dims(**kw)
    assert append(d) == code
    need = ctypes.c_size_t(0)
    assert B.lib().gdn_prefix_attention_workspace_bytes(ctypes.byref(d), 100, 1, 96, ctypes.byref(need)) == code
    assert attend(d) == code


def test_append_arguments():
    d = pool_dims()
    for kw, code in ((dict(A=0), INVALID), (dict(A=5), UNSUPPORTED), (dict(R=80), INVALID), (dict(R=24), UNSUPPORTED),
                     (dict(R=-16), INVALID), (dict(P=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
                     (dict(first=1 << 31), UNSUPPORTED), (dict(q_stride=8), INVALID), (dict(k_stride=132), INVALID),
                     (dict(v_stride=64), INVALID)):
        assert append(d, turn(**kw)) == code, kw
    assert B.lib().gdn_paged_append(ctypes.byref(d), None, *places(14), None) == INVALID
    assert B.lib().gdn_paged_append(None, ctypes.byref(turn()), *places(14), None) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 8, 9, 11, 12, 13):  # q k v wq wk rope table past oq pools
        assert append(d, **{"_%d" % i: None}) == INVALID, i
    one = ctypes.c_void_p((1 << 40) + 8)
    for i in (0, 1, 2, 3, 4, 5, 11, 12, 13):
        assert append(d, **{"_%d" % i: one}) == INVALID, i
    assert append(pool_dims(N=71), _10=None) == INVALID   # 71 tokens are not as many for each of 4
    no_q = pool_dims(Hq=0)
    for at in (dict(), dict(_0=None), dict(_0=None, _11=None), dict(_11=None, _3=None)):
        assert append(no_q, **at) == INVALID, at          # (queries, their output or weights without query heads)


def test_append_overlaps():
    """Outputs on inputs and on each other; keys beside values in one tensor are apart."""
    d = pool_dims()
    p = places(14)
    span = 100 * 2 * 16 * 64 * 2
    size = {0: 70 * 512 * 2, 1: 70 * 128 * 2, 2: 70 * 128 * 2, 3: 256, 4: 256, 5: 50 * 32 * 4, 6: 16, 7: 3 * 70 * 4, 8: 96, 9: 16,
            10: 20}

    def at(i, shift):
        return ctypes.c_void_p(p[i].value + shift)

    for out, n in ((11, 70 * 512 * 2), (12, span), (13, span)):
        for other, m in size.items():
            for shift in (0, (m - 1) // 16 * 16, 16 - n):
                assert append(d, **{"_%d" % out: at(other, shift)}) == INVALID, (out, other, shift)
    assert append(d, _11=at(12, span - 16)) == INVALID
    for shift in (0, 16, 128, span - 16, -16):
        assert append(d, _13=at(12, shift)) == INVALID, shift
    beside = pool_dims(page_stride=2 * 2 * 16 * 64)       # [pages, 2, Hk, page, D]
    for shift in (16, 64 * 2, 2 * 16 * 64 * 2 - 16):
        assert append(beside, _13=at(12, shift)) == INVALID, shift


# ----------------------------------------------------------------------------- attention

def attend(d, prefix=100, max_q=70, max_len=96, ws=1 << 40, **at):
    p = places(10)  # q k v table lens prefix_pages cu o lse ws
    for i, x in at.items():
        p[int(i[1:])] = x
    return B.lib().gdn_prefix_attention(ctypes.byref(d), *p[:6], prefix, p[6], max_q, max_len, 1.0, p[7], p[8], p[9], ws, None)


def test_attention_arguments():
    d = pool_dims()
    lib, need = B.lib(), ctypes.c_size_t(0)

    def query(d, prefix, max_q, max_len):
        return lib.gdn_prefix_attention_workspace_bytes(ctypes.byref(d), prefix, max_q, max_len, ctypes.byref(need))

    assert query(d, 100, 5, 96) == OK and need.value > 0
    for kw, code in ((dict(prefix=-1), INVALID), (dict(max_q=0), INVALID), (dict(max_q=71), INVALID), (dict(max_len=-1), INVALID),
                     (dict(max_len=97), INVALID), (dict(prefix=(1 << 30) + 1), UNSUPPORTED)):
        assert attend(d, **kw) == code, kw
        a = {**dict(prefix=100, max_q=70, max_len=96), **kw}
        assert query(d, a["prefix"], a["max_q"], a["max_len"]) == code, kw
    assert attend(pool_dims(Hq=7)) == INVALID and attend(pool_dims(Hq=0)) == INVALID
    assert attend(pool_dims(N=1 << 25, Hq=4, Hk=1, S=1)) == UNSUPPORTED     # 2^27 rows
    assert attend(pool_dims(N=1 << 20, S=1 << 20), max_q=1 << 20) == UNSUPPORTED  # more items than a launch has
    assert attend(pool_dims(N=71), _6=None) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert attend(d, **{"_%d" % i: None}) == INVALID, i
    one = ctypes.c_void_p((1 << 40) + 8)
    for i in (0, 1, 2, 7, 9):
        assert attend(d, **{"_%d" % i: one}) == INVALID, i
    assert query(d, 100, 70, 96) == OK
    assert attend(d, ws=need.value - 1) == WORKSPACE and attend(d, _9=None) == WORKSPACE
    assert lib.gdn_prefix_attention_workspace_bytes(ctypes.byref(d), 100, 70, 96, None) == INVALID
    assert lib.gdn_prefix_attention_workspace_bytes(None, 100, 70, 96, ctypes.byref(need)) == INVALID


def test_attention_overlaps():
    d = pool_dims()
    p = places(10)
    need = ctypes.c_size_t(0)
    assert B.lib().gdn_prefix_attention_workspace_bytes(ctypes.byref(d), 100, 70, 96, ctypes.byref(need)) == OK
    rows, span = 70 * 8 * 64 * 2, 100 * 2 * 16 * 64 * 2
    size = {0: rows, 1: span, 2: span, 3: 96, 4: 16, 5: 28, 6: 20}
    for out, n in ((7, rows), (8, 70 * 8 * 4), (9, need.value)):
        for other, m in size.items():
            for shift in (0, (m - 1) // 16 * 16, 16 - n // 16 * 16):
                assert attend(d, **{"_%d" % out: ctypes.c_void_p(p[other].value + shift)}) == INVALID, (out, other, shift)
    for a, b in ((7, 8), (7, 9), (8, 9)):
        assert attend(d, **{"_%d" % a: p[b]}) == INVALID


def test_nothing_to_do():
    """No tokens: nothing is launched, whatever the places."""
    assert append(pool_dims(N=0), _0=None, _1=None, _2=None, _11=None, _12=None, _13=None) == OK
    assert attend(pool_dims(N=0), max_q=0, _0=None, _1=None, _2=None, _7=None, _9=None, ws=0) == OK
    assert axes_fwd(axes_dims(T=0), _0=None, _1=None, _7=None, _8=None) == OK


# --------------------------------------------------------------------------- the binding

def test_binding_refuses_on_the_cpu():
    z = torch.zeros
    q, k = z((2, 3, 4, 64)), z((2, 3, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        B.norm_rope_axes(q, k)
    with pytest.raises(ValueError, match="both, or neither"):
        B.norm_rope_axes(q, k, z((64,)))
    pools = z((5, 2, 16, 64)), z((5, 2, 16, 64))
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        B.paged_append(z((3, 4, 64)), z((3, 2, 64)), z((3, 2, 64)), *pools, z((3, 2), **i32), z((3,), **i32))
    with pytest.raises(ValueError, match="GPU"):
        B.prefix_attention(z((3, 4, 64)), *pools, z((3, 2), **i32), z((3,), **i32))


def test_short_way_declines_what_it_does_not_know():
    """Anything but tensors of the GPU, too few arguments, none at all: left to binding.py."""
    if B._calls is None:
        pytest.skip("not built")
    for f in (B._calls.norm_rope_axes, B._calls.norm_rope_axes_bwd, B._calls.paged_append, B._calls.prefix_attention):
        for args in ((), (None,), (torch.zeros((2, 3, 4, 64)),) * 12, (1, 2.0, "x"), (torch.zeros((3, 4, 64)),) * 18, (None,) * 18):
            assert f(*args) is NotImplemented


def test_axis_maps():
    assert B.axis_map((2, 1, 1), device="cpu").tolist() == [0, 0, 1, 2]
    assert B.axis_map((3, 1, 2), cycle=True, device="cpu").tolist() == [0, 1, 2, 0, 2, 0]
    assert B.axis_map((0, 2), device="cpu").tolist() == [1, 1] and B.axis_map((), device="cpu").numel() == 0
