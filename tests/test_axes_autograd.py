"""What NormRopeAxes keeps for its backward pass: without the norm neither queries nor keys,
which its VJP does not read."""
import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B


def kept(f):
    """f's result and the tensors that its graph holds."""
    held = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t) or t, lambda t: t):
        y = f()
    return y, held


@pytest.mark.parametrize("norm", [False, True])
def test_kept(monkeypatch, norm):
    """The entries replaced: no GPU."""
    given = {}
    monkeypatch.setattr(B, "norm_rope_axes", lambda q, k, *a, **kw: (q.clone(), k.clone()))

    def bwd(q, k, wq, wk, rope, axis, pos, dyq, dyk, **kw):
        given.update(q=q, k=k, dyq=dyq, dyk=dyk)
        return dict(dq=dyq, dk=dyk, dwq=wq, dwk=wk)
    monkeypatch.setattr(B, "norm_rope_axes_bwd", bwd)
    q, k = torch.randn(1, 3, 2, 8, requires_grad=True), torch.randn(1, 3, 1, 8, requires_grad=True)
    w = [torch.randn(8, requires_grad=True) for _ in range(2)] if norm else [None, None]
    rope, axis, pos = torch.randn(4, 8), torch.zeros(4, dtype=torch.uint8), torch.zeros((1, 1, 3), dtype=torch.int32)
    (a, b), held = kept(lambda: B.NormRopeAxes.apply(q, k, *w, rope, axis, pos))
    at = {t.data_ptr() for t in held}
    assert {rope.data_ptr(), axis.data_ptr(), pos.data_ptr()} <= at
    assert (q.data_ptr() in at) == (k.data_ptr() in at) == norm
    (2 * a.sum() + 3 * b.sum()).backward()
    assert torch.equal(q.grad, torch.full_like(q, 2.0)) and torch.equal(k.grad, torch.full_like(k, 3.0))
    assert given["q"].shape == q.shape and given["k"].shape == k.shape
    if norm:
        assert torch.equal(given["q"], q) and torch.equal(given["k"], k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_without_norm(dtype, interleaved, packed):
    """The VJP's of the queries and keys, packed or dense; queries that are overwritten
    behind the forward are no matter."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, 5, 6, 64), generator=g, device="cuda").to(dtype)
    leaf = x.clone().requires_grad_()
    q, k = leaf[:, :, :4], leaf[:, :, 4:]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    rope, axis = B.rope_table(30, 32), B.axis_map([8, 8])
    pos = torch.randint(0, 30, (2, 2, 5), generator=g, device="cuda", dtype=torch.int32)
    a, b = B.NormRopeAxes.apply(q, k, None, None, rope, axis, pos, 1e-6, 0.0, interleaved)
    dyq, dyk = torch.randn(a.shape, generator=g, device="cuda").to(dtype), torch.randn(b.shape, generator=g, device="cuda").to(dtype)
    with torch.no_grad():
        leaf.zero_()
    torch.autograd.backward((a, b), (dyq, dyk))
    ref = B.norm_rope_axes_bwd(x[:, :, :4], x[:, :, 4:], None, None, rope, axis, pos, dyq, dyk, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(leaf.grad[:, :, :4], ref["dq"]) and torch.equal(leaf.grad[:, :, 4:], ref["dk"])
