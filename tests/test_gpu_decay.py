"""The decay operator (gdn_decay_fwd, gdn_decay_bwd, through the binding)
against a 64-bit reference that goes one step after the other, with the bounds
derived in decay_reference.py."""
import pytest
import torch

import decay_reference as R
from helpers import say
from linear_attention_recurrence_fwd_amd import binding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()


def make(B, T, Hk, Hv, Dk, Dv, dtype, seed, mask="none", state=True, lg=None):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s, dt=dtype):
        return torch.randn(s, generator=g).to(dt)
    t = dict(q=rnd(B, T, Hk, Dk), k=rnd(B, T, Hk, Dk), v=rnd(B, T, Hv, Dv), dO=rnd(B, T, Hv, Dv),
             lg=-torch.exp2(-8.0 * torch.rand((Hv,), generator=g)),
             state0=rnd(B, Hv, Dk, Dv, dt=F32) if state else None, dS=rnd(B, Hv, Dk, Dv, dt=F32) if state else None)
    if lg is not None:
        t["lg"] = torch.full((Hv,), float(lg)) if not isinstance(lg, (list, tuple)) else torch.tensor(lg)
    m = None
    if mask != "none":
        m = torch.ones((B, T), dtype=torch.uint8)
        n = torch.randint(0, T + 1, (B,), generator=g)
        n[0] = 0  # one row without a valid step
        for b in range(B):
            if mask == "behind":
                m[b, int(n[b]):] = 0
            elif mask == "before":
                m[b, : T - int(n[b])] = 0
        if mask == "some":
            m = (torch.rand((B, T), generator=g) < 0.6).to(torch.uint8)
            m[0] = 0
        bad = m == 0
        for x in ("k", "v"):  # what stands at masked steps is not read
            t[x][bad] = float("nan")
        t["k"][bad.nonzero()[::2].unbind(1)] = float("inf")
    t["mask"] = m
    return t


def up(t):
    return {n: None if x is None else x.cuda() for n, x in t.items()}


def f64(x):
    return None if x is None else x.double()


def run_both(t, algo=binding.ALGO_AUTO, bwd=True, scale=None, tag=""):
    dtype = t["q"].dtype
    rounded = dtype == BF
    c = up(t)
    o, st = binding.decay_fwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"], algo=algo, scale=scale)
    torch.cuda.synchronize()
    k, v = R.clean(f64(t["k"]), f64(t["v"]), t["mask"])
    q, lg, s0 = f64(t["q"]), f64(t["lg"]), f64(t["state0"])
    B, T, Hk, Dk = q.shape
    Dv = v.shape[3]
    sc = None if scale is None else abs(scale)
    ro, rst = R.decay(q, k, v, lg, s0, t["mask"], scale)
    mo, mst = R.decay(q.abs(), k.abs(), v.abs(), lg, None if s0 is None else s0.abs(), t["mask"], sc)
    terms = Dk + Dv + 128 + T
    errs = {"o": R.check("o", o, ro, mo, dtype, terms, rounded),
            "state": R.check("state", st, rst, mst, dtype, terms, False)}
    norm = {"o": R.NORM[rounded], "state": R.NORM[False]}
    if bwd:
        # the VJP knows one algo less
        balgo = binding.ALGO_AUTO if algo == binding.ALGO_SCAN else algo
        g = binding.decay_bwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"], c["dO"], c["dS"], algo=balgo,
                              scale=scale)
        torch.cuda.synchronize()
        dO, dS = f64(t["dO"]), f64(t["dS"])
        rg = R.decay_grads(q, k, v, lg, s0, t["mask"], dO, dS, scale)
        ab = lambda x: None if x is None else x.abs()  # noqa: E731
        mg = R.decay_grads(q.abs(), k.abs(), v.abs(), lg, ab(s0), t["mask"], dO.abs(), ab(dS), sc)
        # dlg: sums over pairs weighted with distances of up to 64 a chunk on top of their own
        like = R.decay_grads(q.abs(), k.abs(), v.abs(), lg, ab(s0), t["mask"], dO.abs(), ab(dS), sc)
        flow = (ro.new_tensor(0.0) + (mo * dO.abs()).sum((0, 1, 3)))
        if dS is not None:
            flow = flow + (mst * dS.abs()).sum((0, 2, 3))
        mg["dlg"] = like["dlg"].abs() + 64 * flow
        for n in ("dq", "dk", "dv"):
            errs[n] = R.check(n, g[n], rg[n], mg[n], dtype, terms + Hk, rounded)
            norm[n] = R.NORM[rounded]
        errs["dstate"] = R.check("dstate", g["dstate"], rg["dstate"], mg["dstate"], dtype, terms, False)
        errs["dlg"] = R.check("dlg", g["dlg"], rg["dlg"], mg["dlg"], dtype, terms, False)
        norm["dstate"] = norm["dlg"] = R.NORM[False]
        if t["mask"] is not None:
            bad = (t["mask"] == 0).cuda()
            assert (g["dv"][bad] == 0).all() and (g["dk"][bad] == 0).all()
    say("[decay %s] %s" % (tag, " ".join("%s=%.1e" % kv for kv in errs.items())))
    for n, e in errs.items():
        assert e <= norm[n], (n, e, norm[n])
    return o, st


SIZES = [  # B, T, Hk, Hv, Dk, Dv
    (1, 2, 1, 1, 8, 8), (2, 31, 1, 2, 16, 8), (2, 33, 2, 2, 64, 32), (1, 64, 2, 4, 64, 64), (3, 65, 1, 1, 40, 72),
    (2, 130, 2, 4, 128, 128), (1, 200, 1, 2, 192, 128), (1, 96, 1, 1, 256, 256), (2, 191, 3, 3, 96, 200),
    (1, 257, 1, 3, 128, 8), (1, 129, 1, 1, 8, 256),
]


@pytest.mark.parametrize("mask", ["none", "behind", "before", "some"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_parity(size, dtype, mask):
    say("[decay] size=%s dtype=%s mask=%s" % (size, dtype, mask))
    run_both(make(*size, dtype, 100 + sum(size), mask), tag="%s %s" % (size, mask))


@pytest.mark.parametrize("algo", [binding.ALGO_SCAN, binding.ALGO_CHUNK, binding.ALGO_CHUNK_TPAR])
@pytest.mark.parametrize("T", [1, 3, 64, 300, 777])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_every_form(dtype, T, algo):
    """The per-step form, one pass and parallel segments, each against the reference."""
    say("[decay form] dtype=%s T=%d algo=%d" % (dtype, T, algo))
    run_both(make(2, T, 2, 4, 64, 48, dtype, 7 + T, "some"), algo, tag="algo %d T %d" % (algo, T))


@pytest.mark.parametrize("lg", [0.0, -1e-4, -3.0, -40.0, -1e30, float("-inf"), 0.01])
def test_decays(lg):
    """No decay, slow and fast ones, a state dropped at every step, growth."""
    t = make(2, 150, 1, 2, 64, 64, F32, 11, "some", lg=lg)
    if lg < -1e3:  # the reference's derivative is 0 * inf there: exp(lg) = 0 exactly, so dlg = 0
        c = up(t)
        g = binding.decay_bwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"], c["dO"], c["dS"])
        assert (g["dlg"] == 0).all()
        run_both(dict(t, lg=torch.full_like(t["lg"], -800.0)), tag="lg -800")
        o, st = binding.decay_fwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"])
        d = torch.full_like(c["lg"], -800.0)
        o2, st2 = binding.decay_fwd(c["q"], c["k"], c["v"], d, c["state0"], c["mask"])
        assert torch.equal(o, o2) and torch.equal(st, st2)
        return
    run_both(t, tag="lg %g" % lg)


@pytest.mark.parametrize("T", [1, 2, 4, 5])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (16, 40), (24, 96), (40, 8), (64, 32), (72, 136), (128, 128), (136, 24), (200, 64),
                                   (248, 256), (256, 200)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_few_steps(dtype, Dk, Dv, T):
    """Calls of a few steps and the first length behind them, at every class of head."""
    say("[decay few] dtype=%s Dk=%d Dv=%d T=%d" % (dtype, Dk, Dv, T))
    run_both(make(3, T, 2, 6, Dk, Dv, dtype, Dk + Dv + T, "some"), bwd=False, tag="few %d %d %d" % (Dk, Dv, T))


@pytest.mark.parametrize("G", [3, 4, 6, 8])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [100, 1300])
def test_groups(T, dtype, G):
    """Value heads that share a key head: their gradients are summed, in twos and one by one."""
    say("[decay groups] dtype=%s G=%d T=%d" % (dtype, G, T))
    run_both(make(2, T, 2, 2 * G, 64, 72, dtype, 17 * G + T, "behind"), tag="G %d T %d" % (G, T))


def test_no_state_and_scale():
    run_both(make(2, 100, 2, 2, 64, 64, BF, 5, state=False), tag="no state")
    run_both(make(1, 100, 1, 2, 64, 64, F32, 6), scale=-2.5, tag="scale")
    run_both(make(1, 100, 1, 2, 64, 64, F32, 6), scale=0.0, tag="scale 0")


@pytest.mark.parametrize("algo", [binding.ALGO_AUTO, binding.ALGO_SCAN, binding.ALGO_CHUNK])
def test_empty(algo):
    t = up(make(2, 0, 1, 2, 64, 32, BF, 3))
    o, st = binding.decay_fwd(t["q"], t["k"], t["v"], t["lg"], t["state0"], None, algo=algo)
    assert o.shape == (2, 0, 2, 32) and torch.equal(st, t["state0"])
    g = binding.decay_bwd(t["q"], t["k"], t["v"], t["lg"], t["state0"], None, t["dO"], t["dS"])
    assert torch.equal(g["dstate"], t["dS"]) and (g["dlg"] == 0).all()


def bits(x):
    """The stored bits (a NaN equals itself)."""
    return x.view(torch.uint8)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_carry_in_place_and_repeats(dtype):
    """Segments carried through the state equal one call; in-place updates and
    repeated calls give the same bits."""
    t = make(2, 260, 1, 2, 64, 96, dtype, 21, "some")
    c = up(t)
    o, st = binding.decay_fwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"])
    o2, st2 = binding.decay_fwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"])
    assert torch.equal(bits(o), bits(o2)) and torch.equal(bits(st), bits(st2))
    s = c["state0"].clone()
    o3, s3 = binding.decay_fwd(c["q"], c["k"], c["v"], c["lg"], s, c["mask"], state_out=s)
    assert s3.data_ptr() == s.data_ptr() and torch.equal(s, st) and torch.equal(bits(o3), bits(o))
    a = binding.decay_bwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"], c["dO"], c["dS"])
    b = binding.decay_bwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"], c["dO"], c["dS"])
    for n in a:
        assert torch.equal(bits(a[n]), bits(b[n])), n
    # prompt, then single tokens in place
    q, k, v = (f64(t[n]) for n in ("q", "k", "v"))
    k, v = R.clean(k, v, t["mask"])
    ro, rst = R.decay(q, k, v, f64(t["lg"]), f64(t["state0"]), t["mask"])
    P = 255
    cut = lambda x, i, j: x[:, i:j].contiguous()  # noqa: E731
    s = c["state0"].clone()
    outs = [binding.decay_fwd(cut(c["q"], 0, P), cut(c["k"], 0, P), cut(c["v"], 0, P), c["lg"], s, cut(c["mask"], 0, P),
                              state_out=s)[0]]
    for i in range(P, 260):
        outs.append(binding.decay_fwd(cut(c["q"], i, i + 1), cut(c["k"], i, i + 1), cut(c["v"], i, i + 1), c["lg"], s,
                                      cut(c["mask"], i, i + 1), state_out=s)[0])
    got = torch.cat(outs, 1).double().cpu()
    assert (got - ro).norm() <= R.NORM[dtype == BF] * ro.norm()
    assert (s.double().cpu() - rst).norm() <= R.NORM[False] * rst.norm()


def test_infinite_cotangents_keep_masked_rows_zero():
    """dO may hold anything: dk and dv of masked steps stay zero."""
    for dtype in (BF, F32):
        t = make(1, 70, 1, 2, 64, 64, dtype, 31, "some")
        t["mask"][0, 10:60:3] = 1
        t["dO"][0, 40] = float("inf")
        c = up(t)
        c["k"].nan_to_num_(0.0, 0.0, 0.0)
        c["v"].nan_to_num_(0.0, 0.0, 0.0)
        g = binding.decay_bwd(c["q"], c["k"], c["v"], c["lg"], c["state0"], c["mask"], c["dO"], c["dS"])
        bad = c["mask"][0] == 0
        assert (g["dk"][0, bad] == 0).all() and (g["dv"][0, bad] == 0).all()


def test_untouched_memory():
    """Rows behind a call's own output stay as they were (outputs in the middle of
    a larger buffer, through the C entry)."""
    import ctypes
    for T, dtype in ((1, BF), (67, BF), (67, F32)):
        t = up(make(1, T, 1, 2, 64, 40, dtype, 41))
        d = binding.make_dims(1, T, 1, 2, 64, 40, dtype)
        n = T * 2 * 40
        buf = torch.full((n + 4096,), 7.0, dtype=dtype, device="cuda")
        st = torch.full((2 * 64 * 40 + 4096,), 7.0, device="cuda")
        wsb = binding._query("gdn_decay_fwd_workspace_bytes", d)
        ws = torch.empty((max(wsb, 1),), dtype=torch.uint8, device="cuda")
        o_at, s_at = buf[2048:], st[2048:]
        rc = binding.lib().gdn_decay_fwd(
            ctypes.byref(d), *[binding._p(t[x]) for x in ("q", "k", "v", "lg")], 1.0, binding._p(t["state0"]), None,
            binding._p(o_at), binding._p(s_at), binding._p(ws), wsb, binding._stream(buf.device))
        torch.cuda.synchronize()
        assert rc == 0
        assert (buf[:2048] == 7).all() and (buf[2048 + n:] == 7).all()
        assert (st[:2048] == 7).all() and (st[2048 + 2 * 64 * 40:] == 7).all()


def test_tensors_past_2_31_elements():
    """v, o, dO and dv of 2.3e9 elements.  With a decay of zero every step stands
    alone: o_t = scale (q_t . k_t) v_t, dv_t = scale (q_t . k_t) dO_t, dq_t = scale
    (dO_t . v_t) k_t, so each row is checked by itself, within the bounds of two
    roundings to bf16 (2^-8 each) and fp32 sums."""
    T, Hv, Dk, Dv = 140_003, 128, 8, 128
    assert T * Hv * Dv > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    q, k, v, dO = r(1, T, 1, Dk), r(1, T, 1, Dk), r(1, T, Hv, Dv), r(1, T, Hv, Dv)
    lg = torch.full((Hv,), float("-inf"), device="cuda")
    say("[decay] T=%d Hv=%d: %d elements" % (T, Hv, T * Hv * Dv))
    o, _ = binding.decay_fwd(q, k, v, lg, None, None, scale=1.0)
    torch.cuda.synchronize()
    qk = (q.float() * k.float()).sum(-1, keepdim=True)
    tol = 2.0 ** -7 + 2.0 ** -16
    for t0 in (0, 64 * 1000, 131_072, T - 200):
        s = slice(t0, t0 + 200)
        ref = qk[:, s] * v[:, s].float()
        assert ((o[:, s].float() - ref).abs() <= tol * ref.abs() + 1e-30).all(), t0
    del o
    gr = binding.decay_bwd(q, k, v, lg, None, None, dO, scale=1.0)
    torch.cuda.synchronize()
    for t0 in (0, 64 * 1000, 131_072, T - 200):
        s = slice(t0, t0 + 200)
        ref = qk[:, s] * dO[:, s].float()
        assert ((gr["dv"][:, s].float() - ref).abs() <= tol * ref.abs() + 1e-30).all(), t0
        dot = (dO[:, s].float() * v[:, s].float()).sum(-1, keepdim=True)
        ref, mag = (dot * k[:, s].float()).sum(2), (dot * k[:, s].float()).abs().sum(2)
        assert ((gr["dq"][:, s, 0].float() - ref).abs() <= tol * mag).all(), t0


def _mixer(B, T, dtype, seed):
    """Inputs of a whole mixer: packed projection, norms, rotation, decay."""
    g = torch.Generator().manual_seed(seed)
    Hk, Hv, D = 2, 4, 64
    rnd = lambda *s, dt=dtype: torch.randn(s, generator=g).to(dt)  # noqa: E731
    return dict(qk=rnd(B, T, 2 * Hk * D), v=rnd(B, T, Hv, D), dO=rnd(B, T, Hv, D), wq=1 + 0.1 * rnd(D, dt=F32),
                wk=1 + 0.1 * rnd(D, dt=F32), rope=binding.rope_table(512, 32, device="cpu"),
                lg=-torch.exp2(-6.0 * torch.rand((Hv,), generator=g)), state0=rnd(B, Hv, D, D, dt=F32)), Hk, Hv, D


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_mixer_together(dtype):
    """The norm with rotation on slices of a packed projection, then the decay
    operator, and gradients through both, against the 64-bit chain.  bf16: q and
    k are rounded between the two (2^-8 each, on top of the operator's own), so
    the normwise bound is twice the operator's."""
    B, T = 2, 150
    t, Hk, Hv, D = _mixer(B, T, dtype, 77)
    c = {n: x.cuda() for n, x in t.items()}
    leaves = [c[n].requires_grad_(True) for n in ("qk", "v", "wq", "wk", "lg", "state0")]
    q, k = (x.reshape(B, T, Hk, D) for x in c["qk"].split(Hk * D, -1))
    q, k = c["qk"][..., : Hk * D].view(B, T, Hk, D), c["qk"][..., Hk * D:].view(B, T, Hk, D)
    qn, kn = binding.NormRope.apply(q, k, c["wq"], c["wk"], c["rope"])
    o, st = binding.DecayAttention.apply(qn, kn, c["v"], c["lg"], c["state0"])
    got = torch.autograd.grad((o.float() * c["dO"].float()).sum() + st.sum(), leaves)
    z = {n: f64(x).requires_grad_(True) for n, x in t.items() if n not in ("dO", "rope")}
    q64, k64 = R.norm_rope(z["qk"][..., : Hk * D].reshape(B, T, Hk, D), z["qk"][..., Hk * D:].reshape(B, T, Hk, D),
                           z["wq"], z["wk"], f64(t["rope"]), None)
    ro, rst = R.decay(q64, k64, z["v"], z["lg"], z["state0"])
    ref = torch.autograd.grad((ro * f64(t["dO"])).sum() + rst.sum(), [z[n] for n in ("qk", "v", "wq", "wk", "lg", "state0")])
    for n, a, b in [("o", o, ro), ("state", st, rst)] + list(zip(("qk", "v", "wq", "wk", "lg", "state0"), got, ref)):
        e = ((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm()).item()
        say("[mixer] %s %s %.1e" % (dtype, n, e))
        assert e <= 2 * R.NORM[dtype == BF], (n, e)


def test_second_derivatives_refused():
    """The VJPs have none of their own: asking for one is an error, not a zero."""
    t, Hk, Hv, D = _mixer(1, 40, F32, 78)
    c = {n: x.cuda() for n, x in t.items()}
    q = c["qk"][..., : Hk * D].reshape(1, 40, Hk, D).contiguous().requires_grad_(True)
    k = c["qk"][..., Hk * D:].reshape(1, 40, Hk, D).contiguous().requires_grad_(True)
    for out in (binding.DecayAttention.apply(q, k, c["v"], c["lg"])[0], binding.NormRope.apply(q, k, c["wq"], c["wk"])[0]):
        g, = torch.autograd.grad((out * out).sum(), [q], create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.sum(), [q])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_graph_stream_and_two_at_once(dtype):
    """Captured into a graph on a side stream and replayed on changed inputs, with
    eager work between the replays; and calls on two streams at a time: the same
    bits as eager calls."""
    t = up(make(2, 300, 2, 4, 64, 64, dtype, 51, "behind"))
    u = up(make(2, 300, 2, 4, 64, 64, dtype, 52, "behind"))
    args = lambda x: (x["q"], x["k"], x["v"], x["lg"], x["state0"], x["mask"])  # noqa: E731

    def work(x):
        o, st = binding.decay_fwd(*args(x))
        g = binding.decay_bwd(*args(x), x["dO"], x["dS"])
        q1 = x["q"][:, :1].contiguous()
        o1, st1 = binding.decay_fwd(q1, x["k"][:, :1].contiguous(), x["v"][:, :1].contiguous(), x["lg"], st, None)
        nq, nk = binding.norm_rope(x["q"], x["q"], w, w, rope)
        n = binding.norm_rope_bwd(x["q"], x["q"], w, w, rope, None, x["q"], x["q"])
        return [o, st, o1, st1, nq, nk] + [g[i] for i in sorted(g)] + [n[i] for i in sorted(n)]
    w = torch.ones((64,), device="cuda")
    rope = binding.rope_table(300, 64)
    want_t, want_u = [x.clone() for x in work(t)], [x.clone() for x in work(u)]
    torch.cuda.synchronize()
    # two streams at a time
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = work(t)
        with torch.cuda.stream(s2):
            b = work(u)
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(a, want_t))
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(b, want_u))
    # a graph, replayed on other inputs
    buf = {n: None if x is None else x.clone() for n, x in t.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work(buf)
    for src, want in ((t, want_t), (u, want_u), (t, want_t), (u, want_u)):
        for n in buf:
            if buf[n] is not None:
                buf[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(out, want))
        work(t)  # eager work between the replays
        torch.cuda.synchronize()
