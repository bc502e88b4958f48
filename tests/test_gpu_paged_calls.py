"""The short way to the rotation's and the paged cache's entries (_calls) gives the long
way's bits, and leaves to it what is out of the ordinary."""
import math

import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def flat(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [z for y in (x.values() if isinstance(x, dict) else x) if y is not None for z in flat(y)]


def both(monkeypatch, f):
    """f's results by the short way (which has to be there) and by the long one."""
    assert B._calls is not None
    a = f()
    monkeypatch.setattr(B, "_calls", None)
    b = f()
    torch.cuda.synchronize()
    a, b = flat(a), flat(b)
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and torch.equal(x, y)
    return a


BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


def rotation(dtype, packed, Hq=4, Hk=2, D=64, R=32, A=2, T=5):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, T, Hq + Hk, D), generator=g, device="cuda").to(dtype)
    q, k = x[:, :, :Hq], x[:, :, Hq:]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    w = [1 + torch.randn(D, generator=g, device="cuda") / 8 for _ in range(2)]
    axis = B.axis_map([R // 4, R // 2 - R // 4], device="cuda") if A == 2 else None
    pos = torch.randint(0, 30, (A, 2, T), generator=g, device="cuda", dtype=torch.int32)
    return q, k, w, B.rope_table(32, R), axis, pos


@BOTH
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
def test_rotation(monkeypatch, dtype, packed, norm, pairs):
    q, k, w, rope, axis, pos = rotation(dtype, packed)
    wq, wk = w if norm else (None, None)
    kw = dict(axis=axis, pos=pos, eps=1e-5, w_offset=0.25, interleaved=pairs)
    y = both(monkeypatch, lambda: B.norm_rope_axes(q, k, wq, wk, rope, **kw))
    monkeypatch.undo()
    both(monkeypatch, lambda: B.norm_rope_axes_bwd(q, k, wq, wk, rope, dyq=y[0], dyk=y[1], **kw))


@BOTH
@pytest.mark.parametrize("ragged", [False, True])
def test_append_and_attention(monkeypatch, dtype, ragged):
    q, k, w, rope, axis, _ = rotation(dtype, True)
    q, k = q.reshape(10, 4, 64), k.reshape(10, 2, 64)
    v = torch.randn((10, 2, 64), device="cuda").to(dtype)
    pos = torch.randint(0, 30, (2, 10), device="cuda", dtype=torch.int32)
    table = torch.tensor([[3, 0], [5, 1]], dtype=torch.int32, device="cuda")
    past = torch.tensor([2, 9], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3, 10], dtype=torch.int32, device="cuda") if ragged else None
    new = [3, 7] if ragged else [5, 5]
    shared = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    old = torch.randn((6, 2, 16, 64), device="cuda").to(dtype)

    def append():
        kp, vp = old.clone(), old.clone()
        out = B.paged_append(q, k, v, kp, vp, table, past, cu, wq=w[0], wk=w[1], rope=rope, axis=axis, pos=pos, eps=1e-5)
        return out, kp, vp

    y, kp, vp = both(monkeypatch, append)
    monkeypatch.undo()
    lens = past + torch.tensor(new, dtype=torch.int32, device="cuda")
    for lse in (False, True):
        both(monkeypatch, lambda: B.prefix_attention(y, kp, vp, table, lens, shared, 20, cu, max_q=7, lse=lse))
        monkeypatch.undo()
    both(monkeypatch, lambda: B.prefix_attention(y, kp, vp, table, lens, None, 0, cu, scale=0.3))


def test_out_of_the_ordinary(monkeypatch):
    """Arguments that the short way does not take end in the long way's results or errors."""
    q, k, w, rope, axis, pos = rotation(torch.float32, False)
    ref = B.norm_rope_axes(q, k, *w, rope, axis=axis, pos=pos)
    for bad in (dict(rope=rope.cpu()), dict(rope=rope.double()), dict(axis=axis.to(torch.int32)), dict(pos=pos[:, :1]),
                dict(q=q.half()), dict(q=q.cpu()), dict(q=q.transpose(-1, -2)), dict(wq=w[0][:-1])):
        a = dict(q=q, k=k, wq=w[0], wk=w[1], rope=rope, axis=axis, pos=pos)
        a.update(bad)
        errors = []
        for short in (B._calls, None):
            monkeypatch.setattr(B, "_calls", short)
            with pytest.raises((TypeError, ValueError, RuntimeError)) as e:
                B.norm_rope_axes(**a)
            errors.append((type(e.value), str(e.value)))
            monkeypatch.undo()
        assert errors[0] == errors[1]
    y = B.norm_rope_axes(q, k, *w, rope, axis=axis, pos=pos)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, y)) and math.isfinite(float(y[0].sum()))
