"""What DecayAttention's backward is called with: losses of the outputs, of the
state, of both, or of neither."""
import pytest
import torch

import decay_reference as R
from helpers import say
from linear_attention_recurrence_fwd_amd import binding


@pytest.mark.parametrize("of_o,of_state", [(True, False), (False, True), (True, True)])
def test_what_the_vjp_is_given(monkeypatch, of_o, of_state):
    """A loss without the state passes no dS_final, one without the outputs zeros (the
    entries replaced: no GPU)."""
    given = {}

    def fwd(q, k, v, lg, state0=None, mask=None, *, scale=None):
        return v.clone(), state0.clone()

    def bwd(q, k, v, lg, state0, mask, dO, dS_final=None, *, scale=None):
        given.update(dO=dO, dS=dS_final)
        return dict(dq=q, dk=k, dv=v, dlg=lg, dstate=state0)
    monkeypatch.setattr(binding, "decay_fwd", fwd)
    monkeypatch.setattr(binding, "decay_bwd", bwd)
    x = [torch.randn(s).requires_grad_(True) for s in ((1, 3, 1, 8), (1, 3, 1, 8), (1, 3, 2, 8), (2,), (1, 2, 8, 8))]
    o, st = binding.DecayAttention.apply(*x)
    (2 * o.sum() * of_o + 3 * st.sum() if of_o and of_state else 2 * o.sum() if of_o else 3 * st.sum()).backward()
    assert torch.equal(given["dO"], torch.full((1, 3, 2, 8), 2.0 if of_o else 0.0)) and given["dO"].is_contiguous()
    if of_state:
        assert torch.equal(given["dS"], torch.full((1, 2, 8, 8), 3.0)) and given["dS"].is_contiguous()
    else:
        assert given["dS"] is None


def test_neither_is_no_call(monkeypatch):
    """A function behind that gives no gradient: the VJP is not called, and there are no gradients."""
    class Stop(torch.autograd.Function):
        @staticmethod
        def forward(ctx, o, st):
            return o.sum() + st.sum()

        @staticmethod
        def backward(ctx, d):
            calls.append("stop")
            return None, None
    calls = []
    monkeypatch.setattr(binding, "decay_fwd", lambda q, k, v, *a, **kw: (v.clone(), a[1].clone()))
    monkeypatch.setattr(binding, "decay_bwd", lambda *a, **kw: calls.append("bwd"))
    x = [torch.randn(s).requires_grad_(True) for s in ((1, 3, 1, 8), (1, 3, 1, 8), (1, 3, 2, 8), (2,), (1, 2, 8, 8))]
    Stop.apply(*binding.DecayAttention.apply(*x)).backward()
    assert calls == ["stop"] and all(t.grad is None for t in x)


def behind_one(*xs):
    """A loss whose gradients of xs are views that begin one element into a larger one."""
    y = torch.cat([xs[0].new_ones(1)] + [x.flatten() for x in xs])
    return (y * torch.arange(y.numel(), device=y.device).to(y.dtype)).sum()


def test_gradients_at_odd_places_are_moved(monkeypatch):
    """The entries take tensors at 16 bytes; autograd's views begin anywhere."""
    given = []

    def decay_bwd(q, k, v, lg, state0, mask, dO, dS_final=None, *, scale=None):
        given.extend([dO, dS_final])
        return dict(dq=q, dk=k, dv=v, dlg=lg, dstate=state0)

    def norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk, **kw):
        given.extend([dyq, dyk])
        return dict(dq=q, dk=k, dwq=wq, dwk=wk)
    monkeypatch.setattr(binding, "decay_fwd", lambda q, k, v, *a, **kw: (v.clone(), a[1].clone()))
    monkeypatch.setattr(binding, "decay_bwd", decay_bwd)
    monkeypatch.setattr(binding, "norm_rope", lambda q, k, *a, **kw: (q.clone(), k.clone()))
    monkeypatch.setattr(binding, "norm_rope_bwd", norm_rope_bwd)
    r = lambda *s: torch.randn(s).requires_grad_(True)  # noqa: E731
    for outs in (binding.DecayAttention.apply(r(1, 3, 1, 8), r(1, 3, 1, 8), r(1, 3, 2, 8), r(2), r(1, 2, 8, 8)),
                 binding.NormRope.apply(r(1, 3, 2, 8), r(1, 3, 1, 8), r(8), r(8))):
        given.clear()
        behind_one(*outs).backward()
        at = 1
        for g, o in zip(given, outs):
            assert g.data_ptr() % 16 == 0 and g.is_contiguous()
            assert torch.equal(g.flatten(), torch.arange(at, at + o.numel(), dtype=torch.float32))
            at += o.numel()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_gradients_at_odd_places(dtype):
    """The same gradients as from a loss that gives them at even places, bit for bit."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt).requires_grad_(True)  # noqa: E731
    q, k, v, lg = r(1, 40, 2, 64), r(1, 40, 2, 64), r(1, 40, 2, 32), r(2, dt=torch.float32)
    w = r(64, dt=torch.float32)
    for outs, leaves in ((lambda: binding.DecayAttention.apply(q, k, v, lg)[:1], (q, k, v, lg)),
                         (lambda: binding.NormRope.apply(q, k, w, w), (q, k, w))):
        got = torch.autograd.grad(behind_one(*outs()), leaves)
        at, loss = 1, 0.0
        for o in outs():
            c = torch.arange(at, at + o.numel(), device="cuda").to(o.dtype).view(o.shape)
            loss, at = loss + (o * c).sum(), at + o.numel()
        want = torch.autograd.grad(loss, leaves)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("of_o,of_state", [(True, False), (False, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_gradients_of_one_output(dtype, of_o, of_state):
    """Against the 64-bit reference, normwise as in decay_reference."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("[decay autograd] %s o=%d state=%d" % (dtype, of_o, of_state))
    g = torch.Generator().manual_seed(5)
    B, T, Hk, Hv, Dk, Dv = 2, 140, 1, 2, 64, 40
    r = lambda *s, dt=dtype: torch.randn(s, generator=g).to(dt)  # noqa: E731
    host = [r(B, T, Hk, Dk), r(B, T, Hk, Dk), r(B, T, Hv, Dv), -torch.rand((Hv,), generator=g), r(B, Hv, Dk, Dv, dt=torch.float32)]
    dO, dS = r(B, T, Hv, Dv), r(B, Hv, Dk, Dv, dt=torch.float32)
    leaves = [x.cuda().requires_grad_(True) for x in host]
    o, st = binding.DecayAttention.apply(*leaves)
    got = torch.autograd.grad((o * dO.cuda()).sum() if of_o else (st * dS.cuda()).sum(), leaves)
    zero = torch.zeros((), dtype=torch.float64)
    ref = R.decay_grads(*[x.double() for x in host], None, dO.double() if of_o else zero, dS.double() if of_state else None)
    for n, a in zip(("dq", "dk", "dv", "dlg", "dstate"), got):
        b = ref[n]
        rounded = dtype == torch.bfloat16 and n in ("dq", "dk", "dv")
        assert (a.double().cpu() - b).norm() <= R.NORM[rounded] * b.norm(), n
