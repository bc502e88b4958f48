"""Plain 64-bit forms of the rotation with several axes, the paged cache and the
attention over it, written for the tests: token by token, key by key, on the CPU.
Beside the values, what bounds a kernel's error at each of them."""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def turns(rope, axis, pos):
    """Complex turns [tokens, R/2] of positions [A, tokens]; NaN where there is no such row."""
    P, R = rope.shape
    t = torch.complex(rope[:, : R // 2].double(), rope[:, R // 2:].double())
    bad = torch.full((1, R // 2), complex(math.nan, math.nan), dtype=torch.complex128)
    t = torch.cat([t, bad])
    out = torch.empty((pos.shape[1], R // 2), dtype=torch.complex128)
    for i in range(R // 2):
        a = 0 if axis is None else int(axis[i])
        p = pos[a].long() if a < pos.shape[0] else torch.full_like(pos[0], -1).long()
        out[:, i] = t[torch.where((p < 0) | (p >= P), P, p), i]
    return out


def pairs(R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(x, z, R, interleaved):
    """x [tokens, H, D] with its pairs turned by z [tokens, R/2]."""
    if not R:
        return x
    one, two = pairs(R, interleaved)
    y = x.clone()
    c, s = z.real[:, None], z.imag[:, None]
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def pair_size(x, R, interleaved):
    """At each channel the size of its pair (what a rotation's rounding goes by)."""
    y = x.abs().clone()
    if R:
        one, two = pairs(R, interleaved)
        n = (x[..., one] ** 2 + x[..., two] ** 2).sqrt()
        y[..., one] = n
        y[..., two] = n
    return y


def norm_turn(x, w, z, R, interleaved, eps, w_offset):
    """(y, bound of its fp32 error): a sum of D squares (D/8 in turn, then a tree), its
    root, a quotient, two products, and three roundings of the rotation: under
    D/16 + 12 half steps of fp32 of the pair's size."""
    x = x.double()
    u = x
    if w is not None:
        r = (x.pow(2).mean(-1, keepdim=True) + eps) ** -0.5
        u = x * r * (w.double() + w_offset)
    return rotate(u, z, R, interleaved), (x.shape[-1] / 16 + 12) * U32 * pair_size(u, R, interleaved)


def norm_turn_vjp(x, w, z, dy, R, interleaved, eps, w_offset):
    """(dx, dw, bound of dx's error, bound of dw's), the errors in fp32."""
    e = rotate(dy.double(), z.conj() if R else None, R, interleaved)
    size = pair_size(dy.double(), R, interleaved)
    if w is None:
        return e, None, 4 * U32 * size, None
    x, w = x.double(), w.double() + w_offset
    D = x.shape[-1]
    r = (x.pow(2).mean(-1, keepdim=True) + eps) ** -0.5
    h, a = x * r, e * w
    dx = r * (a - h * (a * h).mean(-1, keepdim=True))
    big = size * w.abs()
    # two sums over D, the root and the products: each term within D/8 + 20 half steps
    bound = (D / 8 + 20) * U32 * r * (big + h.abs() * (big * h.abs()).mean(-1, keepdim=True))
    rows = x.shape[0] * x.shape[1]
    return dx, (e * h).sum((0, 1)), bound, (rows + D / 16 + 40) * U32 * (size * h.abs()).sum((0, 1))


def places(past, cu, S, N):
    """(sequence, number, place) of every token; sequence None behind the last."""
    out = []
    for t in range(N):
        if cu is None:
            s, i = t // (N // S), t % (N // S)
        else:
            s = next((b for b in range(S) if int(cu[b]) <= t < int(cu[b + 1])), None)
            i = None if s is None else t - int(cu[s])
        out.append((s, i, None if s is None else int(past[s]) + i))
    return out


def append(k, v, k_pages, v_pages, table, past, cu):
    """The pools (64 bits) after turned keys k and values v [N,Hk,D] went in, and which
    rows were written [pages, page]."""
    kp, vp = k_pages.double().clone(), v_pages.double().clone()
    pages, _, page, _ = kp.shape
    S, width = table.shape
    put = torch.zeros((pages, page), dtype=torch.bool)
    for t, (s, _, at) in enumerate(places(past, cu, S, k.shape[0])):
        if s is None or at < 0 or at // page >= width:
            continue
        p = int(table[s, at // page])
        if 0 <= p < pages:
            kp[p, :, at % page], vp[p, :, at % page] = k[t].double(), v[t].double()
            put[p, at % page] = True
    return kp, vp, put


def rows_of(pool, ids, count):
    """The first `count` rows [Hk, count, D] of pages ids; NaN for pages that do not exist."""
    pages, Hk, page, D = pool.shape
    out = torch.full((Hk, count, D), math.nan, dtype=torch.float64)
    for j in range(0, count, page):
        p = int(ids[j // page])
        if 0 <= p < pages:
            n = min(page, count - j)
            out[:, j: j + n] = pool[p, :, :n].double()
    return out


def attention(q, k_pages, v_pages, table, lens, prefix_pages, prefix, cu, scale, max_q=None, max_len=None):
    """(o, lse, bound of o, bound of lse) in 64 bits; NaN rows behind the last sequence.

    The bounds: a score is a sum of D products in fp32, in any order, and one more
    product: within (D + 4) half steps of scale sum |q||k|.  An error d of the scores
    moves a weight by d and the sum by d: 2 d of sum p |v|.  The exponential, the
    weights' and the sums' additions (a tile of 16 at a time, then parts): under
    n / 8 + 64 half steps.  bf16: each weight is rounded once (half a step of bf16),
    and the result once."""
    N, Hq, D = q.shape
    S, width = table.shape
    pages, Hk, page, _ = k_pages.shape
    G = Hq // Hk
    bf = q.dtype == torch.bfloat16
    o = torch.full((N, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((N, Hq), math.nan, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for s in range(S):
        t0, t1 = (s * (N // S), (s + 1) * (N // S)) if cu is None else (int(cu[s]), int(cu[s + 1]))
        n, L = t1 - t0, int(lens[s])
        if L < 0 or (max_len is not None and L > max_len) or (max_q is not None and n > max_q):
            continue
        k = torch.cat([rows_of(k_pages, prefix_pages, prefix), rows_of(k_pages, table[s], L)], 1)
        v = torch.cat([rows_of(v_pages, prefix_pages, prefix), rows_of(v_pages, table[s], L)], 1)
        for i in range(n):
            see = prefix + max(0, L - n + i + 1)
            for h in range(Hq):
                x, kk, vv = q[t0 + i, h].double(), k[h // G, :see], v[h // G, :see]
                if see == 0:
                    o[t0 + i, h], lse[t0 + i, h] = 0.0, -math.inf
                    continue
                a = kk @ x * scale
                lse[t0 + i, h] = torch.logsumexp(a, 0)
                p = torch.softmax(a, 0)
                o[t0 + i, h] = p @ vv
                d = (D + 4) * U32 * abs(scale) * (kk.abs() @ x.abs()).max() + 4 * U32 * a.abs().max()
                sums = (see / 8 + 64) * U32
                size = p @ vv.abs()
                bo[t0 + i, h] = (2 * d + sums + (half_step(torch.bfloat16) if bf else 0.0)) * size \
                    + half_step(q.dtype) * o[t0 + i, h].abs() * 1.01
                bl[t0 + i, h] = d + sums + 4 * U32 * lse[t0 + i, h].abs()
    return o, lse, bo, bl


def within(x, ref, bound, what):
    """x (any type) is ref within bound, NaN and infinities in the same places."""
    x = x.detach().double().cpu()
    assert torch.equal(torch.isnan(x), torch.isnan(ref)), what + ": NaN elsewhere"
    fine = torch.isfinite(ref)
    assert torch.equal(x[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), what + ": infinities"
    over = ((x - ref).abs() - bound)[fine]
    assert over.numel() == 0 or over.max() <= 0, "%s: %g over a bound of %g" % (what, over.max(), bound[fine].max())
