"""The operators for the layers around the delta rule, as measured work.

Two operators, each in the forms a model meets them in:

  decay   linear attention with a decay for each head,
            S_t = g S_{t-1} + k_t v_t^T (a masked step leaves S as it is),
            o_t = scale S_t^T q_t,   g = exp(lg[head]):
          the chunked forward for prompts and training, its backward (dq, dk,
          dv, dlg, dstate) and the recurrent step for single tokens.
  norm    RMS norm of every query and key head with a learned weight and the
          rotation of the first R channels by position, in one pass, forward
          and backward (dq, dk, dwq, dwk).

`own` false: elementary torch operations in 32 bits (sums over whole sequences
in 64), rounded once at the end.  `own` true: this repository's calls.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}
CH = 64  # steps per block of the plain form


# ------------------------------------------------------------------- cases

def _decay(op, B, T, Hk, Hv, Dk, Dv, dtype, mask="none", state=True):
    return dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, mask=mask, state=state)


def _norm(op, B, T, Hq, Hk, D, R, dtype, interleaved=False, packed=False):
    return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, dtype=dtype, interleaved=interleaved, packed=packed)


def listed():
    return [
        # one token of one sequence: what a single user waits for, all latency
        dict(name="decay_step_b1", **_decay("decay_fwd", 1, 1, 16, 32, 128, 128, BF16)),
        # one token of each of 64 sequences: a serving batch, a stream over the states
        dict(name="decay_step_b64", **_decay("decay_fwd", 64, 1, 16, 32, 128, 128, BF16)),
        # a short prompt one step past two chunks, narrow heads
        dict(name="decay_prompt_short", **_decay("decay_fwd", 4, 130, 4, 8, 64, 32, BF16)),
        # the 9B layer shape over 2048 tokens, from a zero state, as in training
        dict(name="decay_fwd_9b", **_decay("decay_fwd", 1, 2048, 16, 64, 192, 128, BF16, state=False)),
        # a batch of prompts of unequal length, padded behind
        dict(name="decay_fwd_padded", **_decay("decay_fwd", 6, 1021, 8, 8, 128, 128, BF16, mask="behind")),
        # one long document with few heads
        dict(name="decay_fwd_32k", **_decay("decay_fwd", 1, 32768, 2, 4, 128, 128, BF16)),
        # 32-bit inputs, ragged
        dict(name="decay_fwd_f32", **_decay("decay_fwd", 2, 777, 4, 8, 128, 64, F32, mask="before")),
        # the backward of the 9B layer shape
        dict(name="decay_bwd_9b", **_decay("decay_bwd", 1, 2048, 16, 64, 192, 128, BF16, state=False)),
        # the backward in 32 bits, ragged and padded
        dict(name="decay_bwd_f32", **_decay("decay_bwd", 2, 515, 4, 4, 64, 96, F32, mask="behind")),
        # queries and keys of 64 single tokens
        dict(name="norm_step_b64", **_norm("norm_fwd", 64, 1, 16, 2, 256, 64, BF16, packed=True)),
        # queries and keys of a prompt, cut out of the packed projection
        dict(name="norm_fwd_2k", **_norm("norm_fwd", 2, 2048, 32, 16, 128, 128, BF16, packed=True)),
        # their gradients, weights' gradients among them
        dict(name="norm_bwd_2k", **_norm("norm_bwd", 2, 2048, 32, 16, 128, 128, BF16)),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 5e12 + w["flops"] / 2e14


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["decay_fwd", "decay_fwd", "decay_step", "decay_bwd", "decay_bwd", "norm_fwd", "norm_bwd"])
        dtype = rng.choice([BF16, BF16, F32])
        if op.startswith("decay"):
            Hk, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4])
            T = 1 if op == "decay_step" else _log_int(rng, 2, 8192)
            case = _decay("decay_bwd" if op == "decay_bwd" else "decay_fwd",
                          _log_int(rng, 1, 96 if T == 1 else 6), T, Hk, Hk * G,
                          8 * _log_int(rng, 2, 32), 8 * _log_int(rng, 1, 32), dtype,
                          rng.choice(["none", "none", "behind", "before", "some"]), rng.random() < 0.6)
        else:
            Hk = rng.choice([1, 2, 4, 8, 16])
            D = 8 * _log_int(rng, 4, 32)
            R = 16 * rng.randint(0, D // 16)
            case = _norm(op, _log_int(rng, 1, 48), _log_int(rng, 1, 4096), Hk * rng.choice([1, 2, 4, 8]), Hk,
                         D, R, dtype, rng.random() < 0.3, rng.random() < 0.5)
        if _cost(case) <= top and work(case)["bytes"] < 2e9:
            return case


# ------------------------------------------------------------------ inputs

def _mask(kind, B, T, g):
    """Valid steps [B, T]: padding behind or before prompts of unequal length
    (one of them may be empty), or single steps left out."""
    dev = g.device
    if kind == "none":
        return None
    n = torch.randint(0, T + 1, (B, 1), generator=g, device=dev)
    n[0, 0] = T
    t = torch.arange(T, device=dev)[None]
    if kind == "behind":
        m = t < n
    elif kind == "before":
        m = t >= T - n
    else:
        m = torch.rand((B, T), generator=g, device=dev) < 0.75
    return m.to(torch.uint8).contiguous()


def rope_table(P, R, device, base=10000.0):
    """cos and sin of the angles of P positions, [P, R] (R/2 cos, R/2 sin)."""
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / max(R, 1))
    a = torch.arange(P, dtype=torch.float64, device=device)[:, None] * f[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def rnd(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    B, T = case["B"], case["T"]
    if case["op"].startswith("decay"):
        Hk, Hv, Dk, Dv = (case[n] for n in ("Hk", "Hv", "Dk", "Dv"))
        s = dict(case=case, q=rnd(B, T, Hk, Dk), k=rnd(B, T, Hk, Dk), v=rnd(B, T, Hv, Dv))
        # slow to fast decays over the heads, moved a little by the seed
        h = torch.arange(1, Hv + 1, device=dev, dtype=torch.float32)
        u = torch.rand((Hv,), generator=g, device=dev)
        s["lg"] = (-torch.exp2(-8.0 * (h - 0.5 + 0.5 * u) / Hv)).contiguous()
        s["state0"] = rnd(B, Hv, Dk, Dv, dtype=torch.float32) if case["state"] else None
        s["mask"] = _mask(case["mask"], B, T, g)
        if case["op"] == "decay_bwd":
            s["dO"] = rnd(B, T, Hv, Dv)
            s["dS"] = rnd(B, Hv, Dk, Dv, dtype=torch.float32) if case["state"] else None
        return s
    Hq, Hk, D, R = (case[n] for n in ("Hq", "Hk", "D", "R"))
    s = dict(case=case)
    if case["packed"]:  # one projection of queries, keys and values
        s["qkv"] = rnd(B, T, (Hq + 2 * Hk) * D)
    else:
        s["q"], s["k"] = rnd(B, T, Hq, D), rnd(B, T, Hk, D)
    s["wq"] = 1 + rnd(D, std=0.1, dtype=torch.float32)
    s["wk"] = 1 + rnd(D, std=0.1, dtype=torch.float32)
    P = max(4096, T)
    s["rope"] = rope_table(P, R, dev) if R else None
    first = torch.randint(0, P - T + 1, (B, 1), generator=g, device=dev)
    s["pos"] = (first + torch.arange(T, device=dev)[None]).to(torch.int32).contiguous()
    if case["op"] == "norm_bwd":
        s["dqn"], s["dkn"] = rnd(B, T, Hq, D), rnd(B, T, Hk, D)
    return s


def _qk(s):
    c = s["case"]
    if "qkv" not in s:
        return s["q"], s["k"]
    B, T, Hq, Hk, D = (c[n] for n in ("B", "T", "Hq", "Hk", "D"))
    x = s["qkv"]
    return x[..., : Hq * D].view(B, T, Hq, D), x[..., Hq * D: (Hq + Hk) * D].view(B, T, Hk, D)


EPS = 1e-6


# -------------------------------------------------- the plain form: decay

def _blocks(x, T, nc):
    """[B, T, H, D] -> [B, H, nc, CH, D] in 32 bits, zeros behind the end."""
    B, _, H, D = x.shape
    y = torch.zeros((B, nc * CH, H, D), dtype=torch.float32, device=x.device)
    y[:, :T] = x
    return y.view(B, nc, CH, H, D).permute(0, 3, 1, 2, 4).contiguous()


def _rows(y, T):
    B, H, nc, _, D = y.shape
    return y.permute(0, 2, 3, 1, 4).reshape(B, nc * CH, H, D)[:, :T]


def _counts(mask, B, T, nc, dev):
    """Valid steps up to and with each step, [B, 1, nc, CH], counted from the
    first, and whether each step is valid."""
    m = torch.zeros((B, nc * CH), dtype=torch.float32, device=dev)
    m[:, :T] = 1.0 if mask is None else (mask != 0).float()
    return m.cumsum(1).view(B, 1, nc, CH), m.view(B, 1, nc, CH)


def _mm(a, b):
    return torch.matmul(a, b.contiguous())


def _attend(q, k, v, lg, n, ok, S0):
    """o_i = sum_{j <= i, valid} e^{lg (n_i - n_j)} (q_i . k_j) v_j + e^{lg n_i} S0^T q_i
    over blocks [B, H, nc, CH, D]; also the final state."""
    B, H, nc, C, Dk = q.shape
    Dv = v.shape[-1]
    L = lg.view(1, H, 1, 1)
    before = n[..., :1] - ok[..., :1]          # valid steps before each block
    after = n[..., -1:]
    k = torch.where(ok[..., None] != 0, k, 0.0)
    v = torch.where(ok[..., None] != 0, v, 0.0)
    low = torch.ones((C, C), dtype=torch.bool, device=q.device).tril()
    D = torch.where(low, torch.exp(L[..., None] * (n[..., :, None] - n[..., None, :])), 0.0)
    o = _mm(_mm(q, k.transpose(-1, -2)) * D, v)
    U = _mm((k * torch.exp(L * (after - n))[..., None]).transpose(-1, -2), v)  # [B,H,nc,Dk,Dv]
    ends = torch.cat([before, after[:, :, -1:]], 2)[..., 0]                     # [B,1,nc+1]
    gap = ends[:, :, :, None] - after[..., 0][:, :, None, :]
    W = torch.where(torch.arange(nc + 1, device=q.device)[:, None] > torch.arange(nc, device=q.device)[None],
                    torch.exp(L * gap.clamp(min=0)), 0.0)                       # [B,H,nc+1,nc]
    S = _mm(W, U.reshape(B, H, nc, Dk * Dv))
    if S0 is not None:
        S = S + torch.exp(L * ends[..., None]) * S0.reshape(B, H, 1, Dk * Dv)
    S = S.view(B, H, nc + 1, Dk, Dv)
    o = o + _mm(q * torch.exp(L * (n - before))[..., None], S[:, :, :nc])
    return o, S[:, :, nc].contiguous()


def _decay_grad(q, k, v, lg, n, ok, S0, dO, dS):
    """d lg: the derivative of o and of the final state in lg, against dO and dS."""
    B, H, nc, C, Dk = q.shape
    Dv = v.shape[-1]
    L = lg.view(1, H, 1, 1)
    before, after = n[..., :1] - ok[..., :1], n[..., -1:]
    k = torch.where(ok[..., None] != 0, k, 0.0)
    v = torch.where(ok[..., None] != 0, v, 0.0)
    low = torch.ones((C, C), dtype=torch.bool, device=q.device).tril()
    dn = n[..., :, None] - n[..., None, :]
    D = torch.where(low, dn * torch.exp(L[..., None] * dn), 0.0)
    X = _mm(q, k.transpose(-1, -2)) * D * _mm(dO, v.transpose(-1, -2))
    total = X.double().sum((2, 3, 4))
    w = torch.exp(L * (after - n))
    U = _mm((k * w[..., None]).transpose(-1, -2), v).reshape(B, H, nc, Dk * Dv)
    V = _mm((k * (w * (after - n))[..., None]).transpose(-1, -2), v).reshape(B, H, nc, Dk * Dv)
    ends = torch.cat([before, after[:, :, -1:]], 2)[..., 0]
    gap = (ends[:, :, :, None] - after[..., 0][:, :, None, :]).clamp(min=0)
    W = torch.where(torch.arange(nc + 1, device=q.device)[:, None] > torch.arange(nc, device=q.device)[None],
                    torch.exp(L * gap), 0.0)
    S, E = _mm(W, U), _mm(W * gap, U) + _mm(W, V)  # the states at the blocks' starts and their derivatives
    if S0 is not None:
        z = torch.exp(L * ends[..., None]) * S0.reshape(B, H, 1, Dk * Dv)
        S, E = S + z, E + z * ends[..., None]
    S, E = S.view(B, H, nc + 1, Dk, Dv), E.view(B, H, nc + 1, Dk, Dv)
    r = n - before
    # e^{lg r} (r S + E)^T q against dO, through the products q^T dO of each block
    y = _mm(q * (torch.exp(L * r) * r)[..., None], S[:, :, :nc]) + _mm(q * torch.exp(L * r)[..., None], E[:, :, :nc])
    total = total + (y.double() * dO.double()).sum((2, 3, 4))
    if dS is not None:
        total = total + (E[:, :, nc].double() * dS.double()).sum((2, 3))
    return total.sum(0).float()


def _plain_decay(s):
    c = s["case"]
    B, T, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    G, dt = Hv // Hk, _TYPES[c["dtype"]]
    scale = Dk ** -0.5
    nc = (T + CH - 1) // CH
    q = _blocks(s["q"], T, nc).repeat_interleave(G, 1) * scale
    k = _blocks(s["k"], T, nc).repeat_interleave(G, 1)
    v = _blocks(s["v"], T, nc)
    n, ok = _counts(s["mask"], B, T, nc, q.device)
    lg = s["lg"]
    if c["op"] == "decay_fwd":
        o, S = _attend(q, k, v, lg, n, ok, s["state0"])
        return _rows(o, T).to(dt), S
    dO = _blocks(s["dO"], T, nc)
    # dq_i: the same sum with (dO, v, k) for (q, k, v) and the state transposed
    S0t = None if s["state0"] is None else s["state0"].transpose(2, 3).contiguous()
    dq, _ = _attend(dO, v, k, lg, n, ok, S0t)
    # dk_j, dv_j: from the last step to the first; a step decays by the valid steps behind it
    f = lambda x: None if x is None else x.flip(2, 3).contiguous()  # noqa: E731
    N = n[:, :, -1:, -1:]
    dk, _ = _reverse(f(v), f(dO), f(q), lg, N - n.flip(2, 3), ok.flip(2, 3), s["dS"], True)
    dv, R = _reverse(f(k), f(q), f(dO), lg, N - n.flip(2, 3), ok.flip(2, 3), s["dS"], False)
    dk, dv = f(dk), f(dv)
    dlg = _decay_grad(q, k, v, lg, n, ok, s["state0"], dO, s["dS"])
    sum_heads = lambda x: x.view(B, Hk, G, nc, CH, -1).sum(2)  # noqa: E731
    return dict(dq=_rows(sum_heads(dq) * scale, T).to(dt), dk=_rows(sum_heads(dk), T).to(dt),
                dv=_rows(dv, T).to(dt), dlg=dlg, dstate=R)


def _reverse(q, k, v, lg, n, ok, S0, transposed):
    """Steps already turned round: n valid steps lie behind each; every step
    gives, and the valid ones (ok) take."""
    B, H, nc, C, Dk = q.shape
    Dv = v.shape[-1]
    L = lg.view(1, H, 1, 1)
    first = torch.cat([torch.zeros_like(n[:, :, :1, :1]), (n + ok)[:, :, :-1, -1:]], 2)  # behind each block
    last = (n + ok)[..., -1:]                                                            # with the block
    low = torch.ones((C, C), dtype=torch.bool, device=q.device).tril()
    D = torch.where(low, torch.exp(L[..., None] * (n[..., :, None] - n[..., None, :])), 0.0)
    q = torch.where(ok[..., None] != 0, q, 0.0)
    o = _mm(_mm(q, k.transpose(-1, -2)) * D, v)
    U = _mm((k * torch.exp(L * (last - n))[..., None]).transpose(-1, -2), v)
    ends = torch.cat([first, last[:, :, -1:]], 2)[..., 0]
    gap = (ends[:, :, :, None] - last[..., 0][:, :, None, :]).clamp(min=0)
    W = torch.where(torch.arange(nc + 1, device=q.device)[:, None] > torch.arange(nc, device=q.device)[None],
                    torch.exp(L * gap), 0.0)
    S = _mm(W, U.reshape(B, H, nc, Dk * Dv))
    if S0 is not None:
        S0 = S0.transpose(2, 3) if transposed else S0
        S = S + torch.exp(L * ends[..., None]) * S0.reshape(B, H, 1, Dk * Dv)
    S = S.view(B, H, nc + 1, Dk, Dv)
    o = o + _mm(q * torch.exp(L * (n - first))[..., None], S[:, :, :nc])
    return o, S[:, :, nc].contiguous()


# --------------------------------------------------- the plain form: norm

def _turn(x, cos, sin, R, interleaved, back=False):
    """The first R channels of [B, T, H, D] turned by the angles [B, T, 1, R/2]."""
    if not R:
        return x
    sin = -sin if back else sin
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y[..., : R // 2], y[..., R // 2: R] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_norm(s):
    c = s["case"]
    R, inter, dt = c["R"], c["interleaved"], _TYPES[c["dtype"]]
    cos = sin = None
    if R:
        t = s["rope"][s["pos"].long()][:, :, None]
        cos, sin = t[..., : R // 2], t[..., R // 2:]

    def forward(x, w):
        x = x.float()
        return _turn(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w, cos, sin, R, inter).to(dt)

    def backward(x, w, dy):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        dy = _turn(dy.float(), cos, sin, R, inter, back=True)
        h, e = x * r, dy * w
        return (r * (e - h * (e * h).mean(-1, keepdim=True))).to(dt), (dy * h).double().sum((0, 1, 2)).float()

    q, k = _qk(s)
    if c["op"] == "norm_fwd":
        return forward(q, s["wq"]), forward(k, s["wk"])
    dq, dwq = backward(q, s["wq"], s["dqn"])
    dk, dwk = backward(k, s["wk"], s["dkn"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


# --------------------------------------------------------------------- run

def run(s):
    c = s["case"]
    if own:
        from linear_attention_recurrence_fwd_amd import binding

        if c["op"] == "decay_fwd":
            return binding.decay_fwd(s["q"], s["k"], s["v"], s["lg"], s["state0"], s["mask"])
        if c["op"] == "decay_bwd":
            return binding.decay_bwd(s["q"], s["k"], s["v"], s["lg"], s["state0"], s["mask"], s["dO"], s["dS"])
        q, k = _qk(s)
        if c["op"] == "norm_fwd":
            return binding.norm_rope(q, k, s["wq"], s["wk"], s["rope"], s["pos"], interleaved=c["interleaved"], eps=EPS)
        return binding.norm_rope_bwd(q, k, s["wq"], s["wk"], s["rope"], s["pos"], s["dqn"], s["dkn"],
                                     interleaved=c["interleaved"], eps=EPS)
    return _plain_decay(s) if c["op"].startswith("decay") else _plain_norm(s)


# -------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    B, T = case["B"], case["T"]
    if case["op"].startswith("decay"):
        Hk, Hv, Dk, Dv = (case[n] for n in ("Hk", "Hv", "Dk", "Dv"))
        qk, val, state = B * T * Hk * Dk, B * T * Hv * Dv, B * Hv * Dk * Dv * 4
        step = 4.0 * B * T * Hv * Dk * Dv  # a state update and a product with the state, per step
        mask = B * T if case["mask"] != "none" else 0
        if case["op"] == "decay_fwd":
            return {"bytes": (2 * qk + 2 * val) * e + mask + state * (2 if case["state"] else 1), "flops": step}
        return {"bytes": (4 * qk + 3 * val) * e + mask + 4 * Hv * 2 + state * (3 if case["state"] else 1),
                "flops": 2.5 * step}
    Hq, Hk, D, R = (case[n] for n in ("Hq", "Hk", "D", "R"))
    x = B * T * (Hq + Hk) * D
    side = B * T * 4 + min(B * T, max(4096, T)) * R * 4 + 8 * D
    if case["op"] == "norm_fwd":
        return {"bytes": 2 * x * e + side, "flops": 7.0 * x}
    return {"bytes": 3 * x * e + side + 8 * D, "flops": 14.0 * x}


# ------------------------------------------------- 64 bits, step by step

def exact(case, seed):
    """Each operator from its definition in 64 bits: the recurrences one step
    after the other, the derivative in lg carried forward beside the state."""
    s = prepare(case, seed)
    return _exact_decay(s) if case["op"].startswith("decay") else _exact_norm(s)


def _exact_decay(s):
    c = s["case"]
    B, T, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    G, dev = Hv // Hk, s["q"].device
    z = dict(dtype=torch.float64, device=dev)
    heads = lambda t: s[t].double().repeat_interleave(G, 2)  # noqa: E731
    q, k, v = heads("q") * Dk ** -0.5, heads("k"), s["v"].double()
    g = torch.exp(s["lg"].double())
    ok = torch.ones((B, T), dtype=torch.bool, device=dev) if s["mask"] is None else s["mask"] != 0
    gate = torch.where(ok[..., None], g[None, None], 1.0)[..., None, None]      # [B,T,Hv,1,1]
    k, v = torch.where(ok[..., None, None], k, 0.0), torch.where(ok[..., None, None], v, 0.0)
    S = torch.zeros((B, Hv, Dk, Dv), **z) if s["state0"] is None else s["state0"].double()
    backward = c["op"] == "decay_bwd"
    if not backward:
        o = torch.empty((B, T, Hv, Dv), **z)
        for t in range(T):
            S = torch.addcmul(gate[:, t] * S, k[:, t, :, :, None], v[:, t, :, None, :])
            o[:, t] = (S * q[:, t, :, :, None]).sum(2)
        return o, S
    dO = s["dO"].double()
    E = torch.zeros_like(S)  # dS / d lg
    dq = torch.empty((B, T, Hv, Dk), **z)
    dlg = torch.zeros((B, Hv), **z)
    live = ok[..., None, None, None].double()
    for t in range(T):
        E = gate[:, t] * (E + live[:, t] * S)
        S = torch.addcmul(gate[:, t] * S, k[:, t, :, :, None], v[:, t, :, None, :])
        dq[:, t] = (S * dO[:, t, :, None, :]).sum(3)
        dlg += ((E * q[:, t, :, :, None]).sum(2) * dO[:, t]).sum(2)
    R = torch.zeros_like(S) if s["dS"] is None else s["dS"].double()
    dlg += (E * R).sum((2, 3))
    dk, dv = torch.empty_like(dq), torch.empty((B, T, Hv, Dv), **z)
    for t in range(T - 1, -1, -1):
        R = torch.addcmul(R, q[:, t, :, :, None], dO[:, t, :, None, :])
        dk[:, t] = live[:, t, :, 0] * (R * v[:, t, :, None, :]).sum(3)
        dv[:, t] = live[:, t, :, 0] * (R * k[:, t, :, :, None]).sum(2)
        R = gate[:, t] * R
    of_group = lambda x: x.view(B, T, Hk, G, -1).sum(3)  # noqa: E731
    return dict(dq=of_group(dq) * Dk ** -0.5, dk=of_group(dk), dv=dv, dlg=dlg.sum(0), dstate=R)


def _exact_norm(s):
    c = s["case"]
    R, D = c["R"], c["D"]
    dev = s["wq"].device
    # the rotation as pairs (first, second) of channels
    i = torch.arange(R // 2, device=dev)
    one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
    if R:
        t = s["rope"].double()[s["pos"].long()]
        turn = torch.complex(t[..., : R // 2], t[..., R // 2:])[:, :, None]

    def rotate(x, z):
        if not R:
            return x
        p = torch.complex(x[..., one], x[..., two]) * z
        x = x.clone()
        x[..., one], x[..., two] = p.real, p.imag
        return x

    def out(x, w):
        x = x.double()
        return rotate(x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double(), turn if R else None)

    def grad(x, w, dy):
        x, w = x.double(), w.double()
        m = x.pow(2).sum(-1, keepdim=True) / D + EPS
        dy = rotate(dy.double(), turn.conj() if R else None)
        dw = (dy * x / m.sqrt()).sum((0, 1, 2))
        a = (dy * w * x).sum(-1, keepdim=True)
        return dy * w / m.sqrt() - x * a / (D * m * m.sqrt()), dw

    q, k = _qk(s)
    if c["op"] == "norm_fwd":
        return out(q, s["wq"]), out(k, s["wk"])
    dq, dwq = grad(q, s["wq"], s["dqn"])
    dk, dwk = grad(k, s["wk"], s["dkn"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
