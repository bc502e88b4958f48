"""The decay operator and its derivatives in 64 bits as recurrences, one step after
the other on the inputs' device (decay_reference's autograd keeps every state, which
long sequences of wide heads have no room for), and the bounds of a whole call."""
import torch

import decay_reference as R


def recurrence(q, k, v, lg, state0, mask, dO=None, dS=None, scale=None):
    """dict(o, state) of fp64 tensors, with dO also dq, dk, dv, dlg, dstate.  Beside the
    state goes its derivative in lg, E <- g (E + S) at a valid step; backward goes R,
    the loss's derivative in the state."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    G = Hv // Hk
    scale = Dk ** -0.5 if scale is None else scale
    z = dict(dtype=torch.float64, device=q.device)
    k, v = R.clean(k, v, mask)
    qh, kh = (x.repeat_interleave(G, 2) for x in (q * scale, k))
    ok = torch.ones((B, T), **z) if mask is None else (mask != 0).to(torch.float64)
    live = ok[..., None, None, None]
    gate = torch.where(live != 0, torch.exp(lg)[None, None, :, None, None], 1.0)
    S = torch.zeros((B, Hv, Dk, Dv), **z) if state0 is None else state0
    E = torch.zeros_like(S)
    o, dq = torch.zeros((B, T, Hv, Dv), **z), torch.zeros((B, T, Hv, Dk), **z)
    dlg = torch.zeros((B, Hv), **z)
    for t in range(T):
        if dO is not None:
            E = gate[:, t] * (E + live[:, t] * S)
        S = gate[:, t] * S + kh[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = torch.matmul(qh[:, t, :, None, :], S)[:, :, 0]
        if dO is not None:
            dq[:, t] = torch.matmul(S, dO[:, t, :, :, None])[..., 0]
            dlg += (torch.matmul(qh[:, t, :, None, :], E)[:, :, 0] * dO[:, t]).sum(-1)
    out = dict(o=o, state=S)
    if dO is None:
        return out
    back = torch.zeros_like(S) if dS is None else dS
    dlg += (E * back).sum((2, 3))
    dk, dv = torch.zeros_like(dq), torch.zeros_like(o)
    for t in range(T - 1, -1, -1):
        back = back + qh[:, t, :, :, None] * dO[:, t, :, None, :]
        dk[:, t] = live[:, t, :, 0] * torch.matmul(back, v[:, t, :, :, None])[..., 0]
        dv[:, t] = live[:, t, :, 0] * torch.matmul(kh[:, t, :, None, :], back)[:, :, 0]
        back = gate[:, t] * back
    of_group = lambda x: x.reshape(B, T, Hk, G, Dk).sum(3)  # noqa: E731
    out.update(dq=of_group(dq) * scale, dk=of_group(dk), dv=dv, dlg=dlg.sum(0), dstate=back)
    return out


def check_call(t, got, scale=None):
    """What a call gave (dict as recurrence's, some of it) for inputs t on the GPU,
    against the recurrences: every value within decay_reference's bound, and normwise:
    bf16 results 2^-8 (see there); fp32 ones five times the root of the terms' number
    (channels and steps) times 2^-24, for the magnitudes that cancel.  Returns the
    normwise errors."""
    dtype = t["q"].dtype
    f64 = lambda x: None if x is None else x.double()  # noqa: E731
    ab = lambda x: None if x is None else x.abs()  # noqa: E731
    k, v = R.clean(f64(t["k"]), f64(t["v"]), t["mask"])
    q, lg, s0, dO, dS = (f64(t[n]) for n in ("q", "lg", "state0", "dO", "dS"))
    bwd = "dq" in got
    ref = recurrence(q, k, v, lg, s0, t["mask"], dO if bwd else None, dS, scale)
    mag = recurrence(ab(q), ab(k), ab(v), lg, ab(s0), t["mask"], ab(dO) if bwd else None, ab(dS),
                     None if scale is None else abs(scale))
    if bwd:  # sums over pairs weighted with distances of up to 64 a chunk on top of their own
        flow = (mag["o"] * dO.abs()).sum((0, 1, 3))
        if dS is not None:
            flow = flow + (mag["state"] * dS.abs()).sum((0, 2, 3))
        mag["dlg"] = mag["dlg"].abs() + 64 * flow
    B, T, Hk, Dk = q.shape
    terms = Dk + v.shape[3] + 128 + T + Hk
    errs = {}
    for n, x in got.items():
        rounded = dtype == torch.bfloat16 and n in ("o", "dq", "dk", "dv")
        errs[n] = R.check(n, x, ref[n].cpu(), mag[n].cpu(), dtype, terms, rounded)
        limit = R.NORM[True] if rounded else 5 * terms ** 0.5 * 2.0 ** -24
        assert errs[n] <= limit, (n, errs[n], limit)
    return errs
