"""Appending to a paged cache and the attention over it have no backward pass: what comes
of inputs that require a gradient says so when one is asked for, instead of having none."""
import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B


def test_a_result_says_so():
    """On the CPU: the results keep their places, with a node behind them where one of the
    inputs requires a gradient, and where gradients are on."""
    x, y = torch.randn(3, requires_grad=True), torch.randn(3)
    a, b = torch.empty(3), torch.empty(2)
    assert B._without_backward("f", (a, b), (y, None)) == (a, b) and not a.requires_grad
    with torch.no_grad():
        assert B._without_backward("f", (a, b), (x, y)) == (a, b) and not a.requires_grad
    r = B._without_backward("f", (a, b), (y, x, None))
    assert r[0] is a and r[1] is b and a.requires_grad and b.requires_grad
    with pytest.raises(NotImplementedError, match="f has no backward pass"):
        (a.sum() * 2).backward()
    B._no_out("f", (y, None))
    with torch.no_grad():
        B._no_out("f", (x,))
    with pytest.raises(RuntimeError, match="no_grad"):
        B._no_out("f", (y, x))


@pytest.mark.gpu
@pytest.mark.parametrize("long_way", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_and_attention(monkeypatch, dtype, long_way):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert B._calls is not None
    if long_way:
        monkeypatch.setattr(B, "_calls", None)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v = rnd(4, 4, 64), rnd(4, 2, 64), rnd(4, 2, 64)
    w = [1 + torch.randn(64, generator=g, device="cuda") / 8 for _ in range(2)]
    table = torch.tensor([[1], [2]], dtype=torch.int32, device="cuda")
    past = torch.tensor([0, 3], dtype=torch.int32, device="cuda")

    def append(q, k, v, w, **kw):
        kp, vp = (torch.zeros((3, 2, 16, 64), dtype=dtype, device="cuda") for _ in range(2))
        return B.paged_append(q, k, v, kp, vp, table, past, wq=w[0], wk=w[1], **kw), kp, vp

    y, kp, vp = append(q, k, v, w)
    attend = lambda q, kp, vp, **kw: B.prefix_attention(q, kp, vp, table, past + 2, **kw)  # noqa: E731
    o, sums = attend(y, kp, vp, lse=True)
    for i in range(5):
        x = [t.detach().clone() for t in (q, k, v, *w)]
        x[i].requires_grad_()
        z, kz, vz = append(*x[:3], x[3:])
        assert torch.equal(z, y) and torch.equal(kz, kp) and torch.equal(vz, vp)
        with pytest.raises(NotImplementedError, match="paged_append"):
            z.float().sum().backward()
        with pytest.raises(RuntimeError, match="no_grad"):
            append(*x[:3], x[3:], out=torch.empty_like(y))
        with torch.no_grad():
            into = torch.empty_like(y)
            z = append(*x[:3], x[3:], out=into)[0]
        assert z is into and torch.equal(z, y) and not z.requires_grad
    for i in range(3):
        x = [t.detach().clone() for t in (y, kp, vp)]
        x[i].requires_grad_()
        for lse in (False, True):
            r = attend(*x, lse=lse)
            r = r if lse else (r,)
            assert all(torch.equal(a, b) for a, b in zip(r, (o, sums)))
            for t in r:
                with pytest.raises(NotImplementedError, match="prefix_attention"):
                    t.float().sum().backward()
        with pytest.raises(RuntimeError, match="no_grad"):
            attend(*x, out=torch.empty_like(o))
        with torch.no_grad():
            r = attend(*x)
        assert torch.equal(r, o) and not r.requires_grad
    torch.cuda.synchronize()
