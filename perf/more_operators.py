"""The operators of the softmax-attention layers that stand between the
recurrent ones, as measured work.

Three operators, each in the forms a model meets them in:

  axes    RMS norm of every query and key head and the rotation of the first R
          channels by positions on several axes (time, height, width): pair i
          turns by the angle of its own axis' position; with and without the
          norm, forward and backward (dq, dk, dwq, dwk).
  append  new tokens of a batch of sequences of unequal length: keys (norm,
          rotation) and values go to their places in a paged cache, queries
          are turned on the way.
  prefix  softmax attention of the new tokens over a prefix that all sequences
          share and over their own pages, causal in these:
            o_i = sum_j p_ij v_j,  p_i = softmax(scale q_i . k_j)
          with j over the prefix and the own keys up to the token itself.

`own` false: elementary torch operations in 32 bits (sums over all rows in 64),
rounded once at the end.  `own` true: this repository's calls.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------- cases

def _axes(op, B, T, Hq, Hk, D, R, dtype, A=3, cycle=False, norm=True, interleaved=False, packed=False):
    return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, dtype=dtype, A=A, cycle=cycle, norm=norm,
                interleaved=interleaved, packed=packed)


def _append(S, q, past, Hq, Hk, D, R, dtype, page, A=0, norm=True, first=0, packed=True):
    """S sequences with past[0] .. past[1] tokens in the cache and q[0] .. q[1] new ones."""
    return dict(op="append", S=S, q_lo=q[0], q_hi=q[1], past_lo=past[0], past_hi=past[1], Hq=Hq, Hk=Hk, D=D, R=R,
                dtype=dtype, page=page, A=A, norm=norm, first=first, packed=packed)


def _prefix(S, q, past, P, Hq, Hk, D, dtype, page, by_token=False):
    return dict(op="prefix", S=S, q_lo=q[0], q_hi=q[1], past_lo=past[0], past_hi=past[1], P=P, Hq=Hq, Hk=Hk, D=D,
                dtype=dtype, page=page, by_token=by_token)


def listed():
    return [
        # queries and keys of 64 single tokens, cut out of the projection
        dict(name="axes_step_b64", **_axes("axes_fwd", 64, 1, 16, 2, 256, 64, BF16, packed=True)),
        # the frames of a video in one sequence, axes in turn from pair to pair
        dict(name="axes_fwd_video", **_axes("axes_fwd", 1, 8192, 32, 8, 128, 128, BF16, cycle=True, packed=True)),
        # their gradients, weights' gradients among them
        dict(name="axes_bwd_video", **_axes("axes_bwd", 1, 8192, 32, 8, 128, 128, BF16, cycle=True)),
        # training in 32 bits without the norm, neighbouring channels as pairs, ragged
        dict(name="axes_bwd_plain_f32", **_axes("axes_bwd", 3, 515, 8, 8, 64, 64, F32, norm=False, interleaved=True)),
        # one token of one sequence: what a single user waits for, all latency
        dict(name="append_step_b1", **_append(1, (1, 1), (777, 777), 16, 2, 256, 64, BF16, 64)),
        # one token of each of 64 sequences behind a shared prefix
        dict(name="append_step_b64", **_append(64, (1, 1), (5, 300), 16, 2, 256, 64, BF16, 64, first=4096)),
        # prompts with images, of unequal length, into empty and half-filled pages
        dict(name="append_prompts", **_append(12, (33, 1500), (0, 100), 32, 8, 128, 128, BF16, 32, A=3)),
        # 32 bits, without the norm
        dict(name="append_f32", **_append(5, (1, 700), (0, 50), 8, 8, 64, 64, F32, 16, norm=False, packed=False)),
        # single tokens of eight users of one system prompt
        dict(name="prefix_step_b8", **_prefix(8, (1, 1), (10, 200), 1000, 16, 2, 256, BF16, 64)),
        # single tokens of 64 users of one long document
        dict(name="prefix_step_b64", **_prefix(64, (1, 1), (100, 2000), 32768, 16, 2, 256, BF16, 64)),
        # the prompts of 16 questions to one document, ragged
        dict(name="prefix_questions", **_prefix(16, (20, 290), (0, 0), 8192, 32, 8, 128, BF16, 32)),
        # drafts of a few tokens, 32 bits, odd sizes
        dict(name="prefix_drafts_f32", **_prefix(5, (4, 4), (1, 333), 2049, 8, 8, 64, F32, 16, by_token=True)),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 5e12 + w["flops"] / (3e14 if case["dtype"] == BF16 else 5e13)


def draw(rng):
    top = {o: max(_cost(c) for c in listed() if c["op"].startswith(o)) for o in ("axes", "append", "prefix")}
    while True:
        op = rng.choice(["axes_fwd", "axes_bwd", "append", "append", "prefix", "prefix", "prefix"])
        dtype = rng.choice([BF16, BF16, F32])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 7, 8])
        D = 8 * _log_int(rng, 4, 32)
        R = 16 * rng.randint(0 if op.startswith("a") else 1, D // 16)
        page = rng.choice([8, 16, 32, 64, 128])
        if op.startswith("axes"):
            case = _axes(op, _log_int(rng, 1, 48), _log_int(rng, 1, 4096), Hq, Hk, D, R, dtype, rng.randint(1, 4),
                         rng.random() < 0.5, rng.random() < 0.7, rng.random() < 0.3, rng.random() < 0.5)
        else:
            S, n = _log_int(rng, 1, 96), rng.choice([1, 1, _log_int(rng, 2, 8), _log_int(rng, 9, 1000)])
            q = (rng.choice([n, max(1, n // 4)]), n)
            past = (0, _log_int(rng, 1, 300 if op == "append" else 1500))
            if op == "append":
                case = _append(S, q, past, Hq, Hk, D, R, dtype, page, rng.choice([0, 2, 3]), rng.random() < 0.7,
                               rng.choice([0, 1000]), rng.random() < 0.5)
            else:
                case = _prefix(S, q, past, rng.choice([0, _log_int(rng, 1, 32768), _log_int(rng, 200, 32768)]), Hq, Hk, D,
                               dtype, page, rng.random() < 0.3)
        if _cost(case) <= top[op[:4] if op.startswith("axes") else op] and work(case)["bytes"] < 2e9:
            if op != "prefix" or _scores(case) < 5e8:  # (the plain form holds them)
                return case


# ------------------------------------------------------------------ inputs

def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly and in no order (the first is hi)."""
    return [hi] + [lo + int((hi - lo + 1) * ((0.6180339887 * s) % 1.0)) for s in range(1, n)]


def _lengths(case):
    """(new tokens, tokens before them) of every sequence."""
    S = case["S"]
    return _spread(S, case["q_lo"], case["q_hi"]), _spread(S, case["past_lo"], case["past_hi"])


def _scores(case):
    n, past = _lengths(case)
    return sum(n) * case["Hq"] * (case["P"] + max(n) + max(past)) + case["S"] * max(n) * case["Hq"] * (max(n) + max(past))


def rope_table(P, R, device, base=10000.0):
    """cos and sin of the angles of P positions, [P, R] (R/2 cos, R/2 sin)."""
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / max(R, 1))
    a = torch.arange(P, dtype=torch.float64, device=device)[:, None] * f[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def axis_map(A, R, cycle, device):
    """The axis of each pair: blocks of pairs, or the axes in turn."""
    i = torch.arange(R // 2, device=device)
    return (i % A if cycle else i * A // max(R // 2, 1)).to(torch.uint8)


def _image_positions(A, N, P, g, device):
    """Positions of N tokens on A axes: frames of rows and columns, from a first one on."""
    t = torch.arange(N, device=device)
    side = max(1, int(math.sqrt(min(N, 1024))))
    at = [t // (side * side), t // side % side, t % side, t]
    first = torch.randint(0, max(1, P - max(side, N)), (A, 1), generator=g, device=device)
    return (torch.stack([at[a] for a in range(A)]) + first).to(torch.int32)


def _pages(counts, g, device):
    """Pages of a pool, given out in no order: one list of counts[i] for each i."""
    order = torch.randperm(sum(counts) + 3, generator=g, device=device).to(torch.int32)
    return order.split([*counts, 3])[: len(counts)], sum(counts) + 3


def _table(lists, device):
    t = torch.full((len(lists), max(1, max(x.numel() for x in lists))), -1, dtype=torch.int32, device=device)
    for row, x in zip(t, lists):
        row[: x.numel()] = x
    return t


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def rnd(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    Hq, Hk, D = (case[n] for n in ("Hq", "Hk", "D"))
    s = dict(case=case)
    if case["op"].startswith("axes"):
        B, T, R, A = (case[n] for n in ("B", "T", "R", "A"))
        if case["packed"]:  # one projection of queries, keys and values
            s["qkv"] = rnd(B, T, (Hq + 2 * Hk) * D)
        else:
            s["q"], s["k"] = rnd(B, T, Hq, D), rnd(B, T, Hk, D)
        P = max(4096, 2 * B * T)
        s["pos"] = _image_positions(A, B * T, P, g, dev).view(A, B, T)
        if case["op"] == "axes_bwd":
            s["dyq"], s["dyk"] = rnd(B, T, Hq, D), rnd(B, T, Hk, D)
    else:
        n, past = _lengths(case)
        N, S, page = sum(n), case["S"], case["page"]
        s["n"], s["past_list"] = n, past
        s["cu"] = None if case["q_lo"] == case["q_hi"] else torch.tensor([0, *n], device=dev).cumsum(0).to(torch.int32)
        counts = [-(-(a + b) // page) for a, b in zip(n, past)]
        P = case.get("P", 0)
        lists, pool = _pages([*counts, -(-P // page)], g, dev)
        s["table"] = _table(lists[:S], dev)
        shape = (pool, page, Hk, D) if case.get("by_token") else (pool, Hk, page, D)
        s["k_pages"], s["v_pages"] = rnd(*shape), rnd(*shape)
        if case.get("by_token"):  # pages of whole tokens
            s["k_pages"], s["v_pages"] = s["k_pages"].transpose(1, 2), s["v_pages"].transpose(1, 2)
        if case["op"] == "prefix":
            s["q"] = rnd(N, Hq, D)
            s["lens"] = torch.tensor([a + b for a, b in zip(n, past)], dtype=torch.int32, device=dev)
            s["prefix"] = lists[S].contiguous() if P else None
            return s
        s["past"] = torch.tensor(past, dtype=torch.int32, device=dev)
        if case["packed"]:
            s["qkv"] = rnd(N, (Hq + 2 * Hk) * D)
        else:
            s["q"], s["k"], s["v"] = rnd(N, Hq, D), rnd(N, Hk, D), rnd(N, Hk, D)
        R, A = case["R"], case["A"]
        P = 16384
        s["pos"] = _image_positions(A, N, P, g, dev) if A else None
    s["rope"] = rope_table(P, R, dev) if R else None
    s["axis"] = axis_map(A, R, case.get("cycle", False), dev) if R and A else None
    s["wq"] = 1 + rnd(D, std=0.1, dtype=torch.float32) if case["norm"] else None
    s["wk"] = 1 + rnd(D, std=0.1, dtype=torch.float32) if case["norm"] else None
    return s


def _qkv(s):
    """Queries, keys and values, cut out of the projection where there is one."""
    if "qkv" not in s:
        return s["q"], s["k"], s.get("v")
    c, x = s["case"], s["qkv"]
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    x = x.unflatten(-1, (Hq + 2 * Hk, D))
    return x[..., :Hq, :], x[..., Hq: Hq + Hk, :], x[..., Hq + Hk:, :]


# ------------------------------------------------------ the plain form: axes

def _turn(x, cos, sin, R, interleaved, back=False):
    """The first R channels of [..., H, D] turned by the angles [..., 1, R/2]."""
    if not R:
        return x
    sin = -sin if back else sin
    y = x.clone()
    one = slice(0, R, 2) if interleaved else slice(0, R // 2)
    two = slice(1, R, 2) if interleaved else slice(R // 2, R)
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * cos - b * sin, b * cos + a * sin
    return y


def _angles(s, pos):
    """cos and sin [tokens..., 1, R/2] of positions [A, tokens...] (or of one axis, [tokens...])."""
    R = s["case"]["R"]
    if not R:
        return None, None
    i = torch.arange(R // 2, device=pos.device)
    at = pos[..., None] if s["axis"] is None else pos[s["axis"].long()].movedim(0, -1)
    at = at.long()
    return s["rope"][at, i][..., None, :], s["rope"][at, R // 2 + i][..., None, :]


def _plain_axes(s):
    c = s["case"]
    R, inter, dt = c["R"], c["interleaved"], _TYPES[c["dtype"]]
    cos, sin = _angles(s, s["pos"])

    def forward(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        return _turn(x, cos, sin, R, inter).to(dt)

    def backward(x, w, dy):
        dy = _turn(dy.float(), cos, sin, R, inter, back=True)
        if w is None:
            return dy.to(dt), None
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        h, e = x * r, dy * w
        return (r * (e - h * (e * h).mean(-1, keepdim=True))).to(dt), (dy * h).double().sum((0, 1, 2)).float()

    q, k, _ = _qkv(s)
    if c["op"] == "axes_fwd":
        return forward(q, s["wq"]), forward(k, s["wk"])
    dq, dwq = backward(q, s["wq"], s["dyq"])
    dk, dwk = backward(k, s["wk"], s["dyk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk) if c["norm"] else dict(dq=dq, dk=dk)


# ---------------------------------------------------- the plain form: append

def _token_places(s):
    """Sequence of every token and its number among the new ones."""
    dev = s["table"].device
    c = s["case"]
    if s["cu"] is None:
        t = torch.arange(c["S"] * c["q_lo"], device=dev)
        return t // c["q_lo"], t % c["q_lo"]
    t = torch.arange(sum(s["n"]), device=dev)
    seq = torch.searchsorted(s["cu"], t, right=True) - 1
    return seq, t - s["cu"][seq]


def _plain_append(s):
    c = s["case"]
    page, dt = c["page"], _TYPES[c["dtype"]]
    q, k, v = _qkv(s)
    seq, i = _token_places(s)
    at = s["past"][seq] + i
    cos, sin = _angles(s, at + c["first"] if s["pos"] is None else s["pos"])

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        return _turn(x, cos, sin, c["R"], False).to(dt)

    where = s["table"][seq, at // page].long()
    s["k_pages"][where, :, at % page] = turned(k, s["wk"])
    s["v_pages"][where, :, at % page] = v
    return turned(q, s["wq"]), s["k_pages"], s["v_pages"]


# ---------------------------------------------------- the plain form: prefix

def _rows_of(pages, lists):
    """Keys or values of the pages [..., M] as [..., Hk, M page, D] in 32 bits."""
    x = pages[lists.clamp(min=0).long()].float().movedim(-3, -4)
    return x.flatten(-3, -2)


def _plain_prefix(s):
    c = s["case"]
    S, P, Hq, Hk, D = (c[n] for n in ("S", "P", "Hq", "Hk", "D"))
    G, n, dt = Hq // Hk, max(s["n"]), _TYPES[c["dtype"]]
    seq, i = _token_places(s)
    N = seq.numel()
    q = s["q"].float().view(N, Hk, G, D) * D ** -0.5
    # own keys, every sequence's queries side by side
    k, v = _rows_of(s["k_pages"], s["table"]), _rows_of(s["v_pages"], s["table"])  # [S, Hk, L, D]
    L = k.shape[2]
    x = torch.zeros((S, Hk, n, G, D), dtype=torch.float32, device=q.device)
    x[seq, :, i] = q
    a = torch.matmul(x.view(S, Hk, n * G, D), k.transpose(-1, -2).contiguous()).view(S, Hk, n, G, L)
    a = a[seq, :, i]                                                              # [N, Hk, G, L]
    count = torch.tensor(s["n"], device=q.device)
    seen = torch.arange(L, device=q.device)[None] <= (s["lens"][seq] - count[seq] + i)[:, None]
    a = torch.where(seen[:, None, None], a, float("-inf"))
    v = torch.where((torch.arange(L, device=q.device)[None] < s["lens"][:, None])[:, None, :, None], v, 0.0)
    rows = q.permute(1, 0, 2, 3).reshape(Hk, N * G, D)
    if P:
        kp, vp = _rows_of(s["k_pages"], s["prefix"])[:, :P], _rows_of(s["v_pages"], s["prefix"])[:, :P]
        b = torch.matmul(rows, kp.transpose(-1, -2).contiguous()).view(Hk, N, G, P).transpose(0, 1)
        a = torch.cat([a, b], -1)
    m = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(m.isinf(), 0.0, m))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    x = torch.zeros((S, Hk, n, G, L), dtype=torch.float32, device=q.device)
    x[seq, :, i] = p[..., :L]
    o = torch.matmul(x.view(S, Hk, n * G, L), v).view(S, Hk, n, G, D)[seq, :, i]
    if P:
        b = p[..., L:].transpose(0, 1).reshape(Hk, N * G, P)
        o = o + torch.matmul(b, vp.contiguous()).view(Hk, N, G, D).transpose(0, 1)
    return o.reshape(N, Hq, D).to(dt)


# --------------------------------------------------------------------- run

def run(s):
    c = s["case"]
    if own:
        from linear_attention_recurrence_fwd_amd import binding

        if c["op"] == "prefix":
            return binding.prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["prefix"], c["P"],
                                            s["cu"], max_q=c["q_hi"])
        q, k, v = _qkv(s)
        if c["op"] == "append":
            return (binding.paged_append(q, k, v, s["k_pages"], s["v_pages"], s["table"], s["past"], s["cu"], wq=s["wq"],
                                         wk=s["wk"], rope=s["rope"], axis=s["axis"], pos=s["pos"], first=c["first"], eps=EPS),
                    s["k_pages"], s["v_pages"])
        if c["op"] == "axes_fwd":
            return binding.norm_rope_axes(q, k, s["wq"], s["wk"], s["rope"], s["axis"], s["pos"],
                                          interleaved=c["interleaved"], eps=EPS)
        g = binding.norm_rope_axes_bwd(q, k, s["wq"], s["wk"], s["rope"], s["axis"], s["pos"], s["dyq"], s["dyk"],
                                       interleaved=c["interleaved"], eps=EPS)
        return g if c["norm"] else dict(dq=g["dq"], dk=g["dk"])
    return _plain_prefix(s) if c["op"] == "prefix" else _plain_append(s) if c["op"] == "append" else _plain_axes(s)


# -------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    Hq, Hk, D = (case[n] for n in ("Hq", "Hk", "D"))
    if case["op"].startswith("axes"):
        N, R, A = case["B"] * case["T"], case["R"], case["A"]
        x = N * (Hq + Hk) * D
        side = A * N * 4 + min(N, 4096) * R * 4 + 8 * D
        if case["op"] == "axes_fwd":
            return {"bytes": 2 * x * e + side, "flops": 7.0 * x}
        return {"bytes": (3 if case["norm"] else 2) * x * e + side + 8 * D, "flops": 14.0 * x}
    n, past = _lengths(case)
    N = sum(n)
    if case["op"] == "append":
        side = N * 4 * max(1, case["A"]) + min(N, 4096) * case["R"] * 4 + 8 * D + 8 * case["S"]
        return {"bytes": 2 * N * (Hq + 2 * Hk) * D * e + side, "flops": 7.0 * N * (Hq + Hk) * D}
    keys = case["P"] + sum(a + b for a, b in zip(n, past))
    pairs = N * case["P"] + sum(a * b + a * (a + 1) // 2 for a, b in zip(n, past))
    return {"bytes": (2 * N * Hq * D + 2 * keys * Hk * D) * e + 4 * (keys // case["page"]), "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------- 64 bits

def exact(case, seed):
    """Each operator from its definition in 64 bits: rotations as products of
    complex numbers, the cache's rows token by token, attention sequence by sequence."""
    s = prepare(case, seed)
    if case["op"] == "prefix":
        return _exact_prefix(s)
    return _exact_append(s) if case["op"] == "append" else _exact_axes(s)


def _pairs(R, interleaved, dev):
    i = torch.arange(R // 2, device=dev)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def _rotated(x, z, R, interleaved):
    if not R:
        return x
    one, two = _pairs(R, interleaved, x.device)
    p = torch.complex(x[..., one], x[..., two]) * z
    x = x.clone()
    x[..., one], x[..., two] = p.real, p.imag
    return x


def _turns(s, pos):
    """Complex numbers [tokens..., 1, R/2] of positions [A, tokens...]."""
    R = s["case"]["R"]
    if not R:
        return None
    t = torch.complex(s["rope"][:, : R // 2].double(), s["rope"][:, R // 2:].double())
    axis = [0] * (R // 2) if s["axis"] is None else s["axis"].tolist()
    return torch.stack([t[pos[a].long(), j] for j, a in enumerate(axis)], -1)[..., None, :]


def _normed(x, w):
    x = x.double()
    return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()


def _exact_axes(s):
    c = s["case"]
    R, D, inter = c["R"], c["D"], c["interleaved"]
    z = _turns(s, s["pos"])
    q, k, _ = _qkv(s)
    if c["op"] == "axes_fwd":
        return _rotated(_normed(q, s["wq"]), z, R, inter), _rotated(_normed(k, s["wk"]), z, R, inter)

    def grad(x, w, dy):
        dy = _rotated(dy.double(), z.conj() if R else None, R, inter)
        if w is None:
            return dy, None
        x, w = x.double(), w.double()
        m = x.pow(2).sum(-1, keepdim=True) / D + EPS
        a = (dy * w * x).sum(-1, keepdim=True)
        return dy * w / m.sqrt() - x * a / (D * m * m.sqrt()), (dy * x / m.sqrt()).sum((0, 1, 2))

    dq, dwq = grad(q, s["wq"], s["dyq"])
    dk, dwk = grad(k, s["wk"], s["dyk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk) if c["norm"] else dict(dq=dq, dk=dk)


def _exact_append(s):
    c = s["case"]
    seq = [b for b, m in enumerate(s["n"]) for _ in range(m)]
    at = [p + i for p, m in zip(s["past_list"], s["n"]) for i in range(m)]
    table = s["table"].tolist()
    dev = s["table"].device
    page = torch.tensor([table[b][a // c["page"]] for b, a in zip(seq, at)], device=dev)
    row = torch.tensor([a % c["page"] for a in at], device=dev)
    pos = s["pos"] if s["pos"] is not None else torch.tensor([at], device=dev) + c["first"]
    z = _turns(s, pos)
    q, k, v = _qkv(s)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    kp[page, :, row] = _rotated(_normed(k, s["wk"]), z, c["R"], False)
    vp[page, :, row] = v.double()
    return _rotated(_normed(q, s["wq"]), z, c["R"], False), kp, vp


def _exact_prefix(s):
    c = s["case"]
    P, Hq, Hk, D = (c[n] for n in ("P", "Hq", "Hk", "D"))
    G = Hq // Hk

    def keys(pages, ids, count):
        return pages[ids[: -(-count // c["page"])].long()].double().transpose(0, 1).reshape(Hk, -1, D)[:, :count]

    shared = [keys(x, s["prefix"], P) for x in (s["k_pages"], s["v_pages"])] if P else None
    out, begin = [], 0
    for b, (m, past) in enumerate(zip(s["n"], s["past_list"])):
        q = s["q"][begin: begin + m].double().view(m, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * m, D)
        begin += m
        k, v = (keys(x, s["table"][b], past + m) for x in (s["k_pages"], s["v_pages"]))
        if P:
            k, v = torch.cat([shared[0], k], 1), torch.cat([shared[1], v], 1)
        a = torch.matmul(q, k.transpose(1, 2).contiguous()) / math.sqrt(D)
        last = P + past + torch.arange(m, device=q.device).repeat(G)
        a = a.masked_fill(torch.arange(k.shape[1], device=q.device)[None] > last[:, None], float("-inf"))
        o = torch.matmul(torch.softmax(a, -1), v)
        out.append(o.view(Hk, G, m, D).permute(2, 0, 1, 3).reshape(m, Hq, D))
    return torch.cat(out)
