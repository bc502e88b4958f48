"""The decay operator and the query/key norm with rotation on the CPU: sizes and
refusals of the C entries (no pointer here is ever dereferenced), refusals of the
binding, and the 64-bit references against central differences."""
import ctypes

import pytest
import torch

import decay_reference as R
from linear_attention_recurrence_fwd_amd import binding as B

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def ptrs(n):
    return [ctypes.c_void_p(4096 * (i + 1)) for i in range(n)]


def size(fn, d):
    out = ctypes.c_size_t(0)
    return getattr(B.lib(), fn)(ctypes.byref(d), ctypes.byref(out)), out.value


@pytest.mark.parametrize("dims,code", [
    ((0, 8, 1, 1, 64, 64), INVALID), ((1, -1, 1, 1, 64, 64), INVALID), ((1, 8, 2, 3, 64, 64), INVALID),
    ((1, 8, 1, 1, 0, 64), INVALID), ((1, 8, 1, 1, 12, 64), UNSUPPORTED), ((1, 8, 1, 1, 64, 260), UNSUPPORTED),
    ((1, 8, 1, 1, 264, 64), UNSUPPORTED), ((1, (1 << 30) + 1, 1, 1, 64, 64), UNSUPPORTED),
    ((1, 8, 1, 1 << 20, 64, 64), UNSUPPORTED), ((1 << 40, 8, 1, 1, 64, 64), UNSUPPORTED),
    ((1 << 21, 8, 1, 64, 64, 64), UNSUPPORTED),
])
def test_decay_bad_dims(dims, code):
    for fn in ("gdn_decay_fwd_workspace_bytes", "gdn_decay_bwd_workspace_bytes"):
        assert size(fn, B.make_dims(*dims, B.GDN_BF16))[0] == code


def test_decay_sizes():
    for dt in (B.GDN_F32, B.GDN_BF16):
        assert size("gdn_decay_fwd_workspace_bytes", B.make_dims(3, 1, 2, 4, 64, 40, dt)) == (0, 0)  # a single step
        assert size("gdn_decay_fwd_workspace_bytes", B.make_dims(3, 4, 2, 4, 64, 40, dt)) == (0, 0)  # a few
        assert size("gdn_decay_fwd_workspace_bytes", B.make_dims(3, 500, 2, 4, 64, 40, dt, B.ALGO_CHUNK)) == (0, 0)
        assert size("gdn_decay_fwd_workspace_bytes", B.make_dims(3, 500, 2, 4, 64, 40, dt, B.ALGO_SCAN)) == (0, 0)
        n = size("gdn_decay_fwd_workspace_bytes", B.make_dims(1, 32768, 2, 4, 128, 128, dt))
        assert n[0] == 0 and n[1] >= 64 * 4 * 128 * 128 * 4  # 64 segments' states
        # empty sequences and long ones
        assert size("gdn_decay_bwd_workspace_bytes", B.make_dims(3, 0, 2, 4, 64, 40, dt))[0] == 0
        assert size("gdn_decay_bwd_workspace_bytes", B.make_dims(1, 1 << 30, 1, 1, 64, 40, dt))[0] == 0
    assert size("gdn_decay_bwd_workspace_bytes", B.make_dims(1, 64, 1, 1, 64, 64, B.GDN_BF16, B.ALGO_SCAN))[0] == UNSUPPORTED
    assert size("gdn_decay_fwd_workspace_bytes", B.make_dims(1, 64, 1, 1, 64, 64, 5))[0] == UNSUPPORTED
    assert size("gdn_decay_fwd_workspace_bytes", B.make_dims(1, 64, 1, 1, 64, 64, B.GDN_BF16, 9))[0] == INVALID
    assert B.lib().gdn_decay_fwd_workspace_bytes(None, ctypes.byref(ctypes.c_size_t(0))) == INVALID
    assert B.lib().gdn_decay_fwd_workspace_bytes(ctypes.byref(B.make_dims(1, 64, 1, 1, 64, 64, B.GDN_BF16)), None) == INVALID


def test_decay_fwd_rejects_before_launch():
    lib = B.lib()
    d = B.make_dims(1, 2048, 2, 4, 64, 64, B.GDN_BF16)
    need = size("gdn_decay_fwd_workspace_bytes", d)[1]
    assert need > 0

    def call(p, ws, n, dims=d):  # q k v lg | state0 mask o state_out
        return lib.gdn_decay_fwd(ctypes.byref(dims) if dims else None, *p[:4], 1.0, *p[4:], ws, n, None)
    p, ws = ptrs(8), ctypes.c_void_p(1 << 20)
    for i in (0, 1, 2, 3, 6, 7):
        a = list(p)
        a[i] = None
        assert call(a, ws, need) == INVALID, i
    for i in (0, 1, 2, 4, 6, 7):  # 16-byte alignment
        a = list(p)
        a[i] = ctypes.c_void_p(4096 + 8)
        assert call(a, ws, need) == INVALID, i
    assert call(p, ws, need - 1) == WORKSPACE
    assert call(p, None, need) == WORKSPACE
    assert call(p, ctypes.c_void_p((1 << 20) + 4), need) == INVALID
    assert call(p, ws, need, None) == INVALID


def test_decay_bwd_rejects_before_launch():
    lib = B.lib()
    d = B.make_dims(1, 100, 2, 4, 64, 64, B.GDN_F32)
    need = size("gdn_decay_bwd_workspace_bytes", d)[1]
    p, ws = ptrs(14), ctypes.c_void_p(1 << 20)

    def call(a, w, n):  # q k v lg | state0 mask dO dS dq dk dv dlg dstate
        return lib.gdn_decay_bwd(ctypes.byref(d), *a[:4], 1.0, *a[4:13], w, n, None)
    for i in (0, 1, 2, 3, 6, 8, 9, 10, 11, 12):
        a = list(p)
        a[i] = None
        assert call(a, ws, need) == INVALID, i
    for i in (0, 1, 2, 4, 6, 7, 8, 9, 10, 12):
        a = list(p)
        a[i] = ctypes.c_void_p(4096 + 4)
        assert call(a, ws, need) == INVALID, i
    assert call(p, ws, need - 1) == WORKSPACE
    assert call(p, None, need) == WORKSPACE


def spread(n, step):
    return [ctypes.c_void_p((1 << 30) + i * step) for i in range(n)]


@pytest.mark.parametrize("T", [3, 100])
def test_decay_refuses_overlaps(T):
    """Outputs that share bytes with inputs or each other: by all of them, or by the last sixteen."""
    lib, ws = B.lib(), ctypes.c_void_p(1 << 20)
    d = B.make_dims(1, T, 2, 4, 64, 64, B.GDN_F32)
    key, val, state = T * 2 * 64 * 4, T * 4 * 64 * 4, 4 * 64 * 64 * 4
    f = spread(8, 1 << 20)  # q k v lg | state0 mask o state_out
    nbytes = {0: key, 1: key, 2: val, 3: 16, 4: state, 6: val, 7: state}
    for out in (6, 7):
        for i in nbytes:
            if i == out:
                continue
            for shift in (0, nbytes[i] - 16, 16 - nbytes[out]):
                if (out, i, shift) == (7, 4, 0):
                    continue  # in place
                a = list(f)
                a[out] = ctypes.c_void_p(f[i].value + shift)
                assert lib.gdn_decay_fwd(ctypes.byref(d), *a[:4], 1.0, *a[4:], ws, 1 << 19, None) == INVALID, (out, i, shift)
    g = spread(13, 1 << 20)  # q k v lg | state0 mask dO dS dq dk dv dlg dstate
    nbytes = {0: key, 1: key, 2: val, 3: 16, 4: state, 6: val, 7: state, 8: key, 9: key, 10: val, 11: 16, 12: state}
    for out in (8, 9, 10, 12):
        for i in nbytes:
            if i == out:
                continue
            for shift in (0, nbytes[i] - 16, 16 - nbytes[out]):
                a = list(g)
                a[out] = ctypes.c_void_p(g[i].value + shift)
                assert lib.gdn_decay_bwd(ctypes.byref(d), *a[:4], 1.0, *a[4:], ws, 1 << 19, None) == INVALID, (out, i, shift)
    for i in (6, 7):  # the workspace
        if T > 4:
            big = B.make_dims(1, 2048, 2, 4, 64, 64, B.GDN_BF16)
            assert lib.gdn_decay_fwd(ctypes.byref(big), *f[:4], 1.0, *f[4:], f[i], 1 << 24, None) == INVALID


def test_norm_refuses_overlaps():
    lib, d = B.lib(), norm_dims(q_stride=6 * 64, k_stride=6 * 64)
    q, k = 6 * 4 * 64 * 2, 6 * 2 * 64 * 2
    f = spread(8, 1 << 20)  # q k wq wk rope pos oq ok
    qs, ks = (5 * 6 + 4) * 64 * 2, (5 * 6 + 2) * 64 * 2
    for out, n in ((6, q), (7, k)):
        for i, m in ((0, qs), (1, ks), (13 - out, k if out == 6 else q)):
            for shift in (0, m - 16, 16 - n):
                a = list(f)
                a[out] = ctypes.c_void_p(f[i].value + shift)
                assert lib.gdn_norm_rope_fwd(ctypes.byref(d), *a, None) == INVALID, (out, i, shift)
    g, ws = spread(12, 1 << 20), ctypes.c_void_p(1 << 20)  # q k wq wk rope pos dyq dyk dq dk dwq dwk
    for out, n in ((8, q), (9, k)):
        for i, m in ((0, qs), (1, ks), (6, q), (7, k), (17 - out, k if out == 8 else q)):
            for shift in (0, m - 16, 16 - n):
                a = list(g)
                a[out] = ctypes.c_void_p(g[i].value + shift)
                assert lib.gdn_norm_rope_bwd(ctypes.byref(d), *a, ws, 1 << 19, None) == INVALID, (out, i, shift)


def norm_dims(**kw):
    v = dict(B=2, T=3, Hq=4, Hk=2, D=64, R=32, P=16, q_stride=0, k_stride=0, dtype=B.GDN_BF16, interleaved=0, eps=1e-6,
             w_offset=0.0)
    v.update(kw)
    return B.NormDims(*[v[n] for n, _ in B.NormDims._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(D=0), INVALID),
    (dict(D=12), UNSUPPORTED), (dict(D=520), UNSUPPORTED), (dict(R=24), UNSUPPORTED), (dict(R=80), INVALID),
    (dict(R=-16), INVALID), (dict(P=-1), INVALID), (dict(q_stride=255), INVALID), (dict(k_stride=64), INVALID),
    (dict(q_stride=260), INVALID), (dict(dtype=4), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(B=1 << 20, T=1 << 20), UNSUPPORTED),
])
def test_norm_bad_dims(kw, code):
    d = norm_dims(**kw)
    out = ctypes.c_size_t(0)
    assert B.lib().gdn_norm_rope_bwd_workspace_bytes(ctypes.byref(d), ctypes.byref(out)) == code
    p = ptrs(13)
    assert B.lib().gdn_norm_rope_fwd(ctypes.byref(d), *p[:8], None) == code
    assert B.lib().gdn_norm_rope_bwd(ctypes.byref(d), *p[:12], p[12], 1 << 30, None) == code


def test_norm_rejects_before_launch():
    lib, d = B.lib(), norm_dims()
    p = ptrs(8)  # q k wq wk rope pos oq ok
    for i in (0, 1, 2, 3, 4, 6, 7):
        a = list(p)
        a[i] = None
        assert lib.gdn_norm_rope_fwd(ctypes.byref(d), *a, None) == INVALID, i
        a[i] = ctypes.c_void_p(4096 + 8)
        assert lib.gdn_norm_rope_fwd(ctypes.byref(d), *a, None) == INVALID, i
    out = ctypes.c_size_t(0)
    assert lib.gdn_norm_rope_bwd_workspace_bytes(ctypes.byref(d), ctypes.byref(out)) == 0 and out.value > 0
    p, ws = ptrs(12), ctypes.c_void_p(1 << 20)  # q k wq wk rope pos dyq dyk dq dk dwq dwk
    for i in (0, 1, 2, 3, 4, 6, 7, 8, 9, 10, 11):
        a = list(p)
        a[i] = None
        assert lib.gdn_norm_rope_bwd(ctypes.byref(d), *a, ws, out.value, None) == INVALID, i
    assert lib.gdn_norm_rope_bwd(ctypes.byref(d), *p, ws, out.value - 1, None) == WORKSPACE
    assert lib.gdn_norm_rope_bwd(ctypes.byref(d), *p, None, out.value, None) == WORKSPACE


def test_token_strides():
    """Slices of a packed projection have a stride; views whose tokens are not
    evenly spaced, or lie on each other, are refused."""
    x = torch.zeros((2, 5, 6 * 64))
    assert B._token_stride(x[..., :256].view(2, 5, 4, 64), "q") == 6 * 64
    assert B._token_stride(x.view(2, 5, 6, 64), "q") == 0
    assert B._token_stride(x[:, :1, :256].view(2, 1, 4, 64), "q") == 5 * 6 * 64
    for bad in (x[:, :3, :256].view(2, 3, 4, 64), torch.zeros((1, 1, 4, 64)).expand(3, 1, 4, 64),
                torch.zeros((1, 1, 4, 64)).expand(1, 3, 4, 64), x.view(2, 5, 6, 64)[:, :, ::2],
                x.view(2, 5, 6, 64)[..., :32], x.view(2, 5, 6, 64).transpose(1, 2)):
        with pytest.raises(ValueError):
            B._token_stride(bad, "q")


def test_binding_refuses_cpu_tensors():
    z = torch.zeros((1, 2, 1, 64))
    with pytest.raises(ValueError):
        B.decay_fwd(z, z, z, torch.zeros((1,)))
    with pytest.raises(ValueError):
        B.norm_rope(z, z, torch.zeros((64,)), torch.zeros((64,)))


def test_rope_table():
    t = B.rope_table(300, 8, base=100.0, device="cpu")
    a = torch.arange(300, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(4, dtype=torch.float64) / 4)
    assert torch.equal(t, torch.cat([torch.cos(a), torch.sin(a)], 1).float())
    assert B.rope_table(5, 0, device="cpu").shape == (5, 0)


def test_references_against_differences():
    """The references' gradients (which the GPU's are held to) against central
    differences of their forwards."""
    g = torch.Generator().manual_seed(1)
    d = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(True)  # noqa: E731
    m = torch.tensor([[1, 0, 1, 1, 0], [0, 0, 0, 0, 0]], dtype=torch.uint8)
    lg = (-torch.rand(2, generator=g, dtype=torch.float64)).requires_grad_(True)
    assert torch.autograd.gradcheck(lambda *a: R.decay(*a, m), (d(2, 5, 1, 3), d(2, 5, 1, 3), d(2, 5, 2, 2), lg, d(2, 2, 3, 2)))
    rope = B.rope_table(9, 4, device="cpu").double()
    pos = torch.tensor([[3, 8, 0]])
    for inter in (False, True):
        assert torch.autograd.gradcheck(
            lambda *a: R.norm_rope(*a, rope, pos, 1e-6, 0.5, inter), (d(1, 3, 2, 6), d(1, 3, 1, 6), d(6), d(6)))
