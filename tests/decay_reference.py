"""Plain 64-bit references, on the CPU, of the decay operator (one step after
the other; gradients by torch's autograd through those steps) and of the
query/key norm with rotation, and the bounds their tests hold the GPU to.

Bounds.  With u = 2^-8 for bf16 (half a step relative to the value) and 2^-24
for fp32, every product that a kernel rounds to the tensors' type, and every
fp32 sum of n terms, is off by at most u (n 2^-24) times the sum of the terms'
magnitudes.  Those magnitudes are bounded by the same operator run on |q|, |k|,
|v|, |state| (`magnitude`), so an output o is off by at most
    u |o| + (2 u + n 2^-24) magnitude
(its own rounding; the rounding of the products with the chunk's steps and with
the state; the sums), n = Dk + Dv + 64 + T for the sums over channels, steps and
chunks plus 64 for the exponentials (each at most 2^-22 |x| e^-|x| off).  fp32
tensors are not rounded in between: there u counts only for the output.
"""
import torch


def decay(q, k, v, lg, state0=None, mask=None, scale=None):
    """o [B,T,Hv,Dv] and the final state, all fp64, differentiable."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    G = Hv // Hk
    scale = Dk ** -0.5 if scale is None else scale
    S = torch.zeros((B, Hv, Dk, Dv), dtype=torch.float64) if state0 is None else state0
    g = torch.exp(lg).view(1, Hv, 1, 1)
    out = []
    for t in range(T):
        kt, qt = k[:, t].repeat_interleave(G, 1), q[:, t].repeat_interleave(G, 1)
        new = g * S + kt[..., None] * v[:, t, :, None, :]
        if mask is not None:
            new = torch.where((mask[:, t] != 0).view(B, 1, 1, 1), new, S)
        S = new
        out.append(scale * (S * qt[..., None]).sum(2))
    return (torch.stack(out, 1) if T else torch.zeros((B, 0, Hv, Dv), dtype=torch.float64)), S


def decay_grads(q, k, v, lg, state0, mask, dO, dS, scale=None):
    """Gradients of <o, dO> + <state, dS>; masked k and v are taken as zeros
    (they are not read into anything)."""
    if mask is not None:
        m = (mask != 0)[..., None, None]
        k, v = torch.where(m, k, 0.0), torch.where(m, v, 0.0)
    B, T, Hk, Dk = q.shape
    s0 = state0 if state0 is not None else torch.zeros((B, v.shape[2], Dk, v.shape[3]), dtype=torch.float64)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, lg, s0)]
    o, S = decay(*leaves, mask, scale)
    loss = (o * dO).sum()
    if dS is not None:
        loss = loss + (S * dS).sum()
    loss = loss + 0.0 * sum(x.sum() for x in leaves)  # every leaf has a gradient, also with T = 0
    gs = torch.autograd.grad(loss, leaves)
    return dict(zip(("dq", "dk", "dv", "dlg", "dstate"), gs))


def clean(k, v, mask):
    if mask is None:
        return k, v
    m = (mask != 0)[..., None, None]
    return torch.where(m, k, 0.0), torch.where(m, v, 0.0)


def check(name, got, ref, magnitude, dtype, terms, rounded):
    """got against ref within the bound above; `rounded`: stored in bf16."""
    got, ref = got.detach().double().cpu(), ref.detach()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not ref.numel():
        return 0.0
    assert torch.isfinite(got).all(), name
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    own = (2.0 ** -8 if rounded else 2.0 ** -24) * ref.abs()
    bound = own + (2 * u * (1 if rounded else 0) + terms * 2.0 ** -24) * magnitude.detach() + 1e-37
    worst = ((got - ref).abs() / bound).max().item()
    assert worst <= 1.0, "%s: %.2f times its bound" % (name, worst)
    n = ref.norm().item()
    return (got - ref).norm().item() / n if n else 0.0


# Normwise (2-norm), where the errors of the single products are independent: a
# rounding to bf16 has a root-mean-square error of at most 2^-8 / sqrt(3), and
# three of them meet in an output (its own, the products with the steps, the
# products with the state), 2^-8 together.  fp32 results: sums of about a
# thousand terms, sqrt(1000) 2^-24 = 2e-6, taken five times for the magnitudes
# that cancel.
NORM = {True: 2.0 ** -8, False: 1e-5}


def norm_rope(q, k, wq, wk, rope, pos, eps=1e-6, w_offset=0.0, interleaved=False):
    """(q, k) fp64, differentiable in q, k, wq, wk."""
    T = q.shape[1]

    def one(x, w):
        B = x.shape[0]
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (w + w_offset)
        if rope is None or rope.shape[1] == 0:
            return y
        R = rope.shape[1]
        p = torch.arange(T)[None].expand(B, T) if pos is None else pos.long()
        c, s = rope[p][:, :, None, : R // 2], rope[p][:, :, None, R // 2:]
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., : R // 2], y[..., R // 2: R])
        y1, y2 = a * c - b * s, b * c + a * s
        front = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
        return torch.cat([front, y[..., R:]], -1)
    return one(q, wq), one(k, wk)
