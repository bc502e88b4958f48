"""The norm and rotation with positions on several axes against 64 bits: forward and
VJP, every class of head sizes, axes in blocks and in turn, both pairings, with and
without the norm, packed and dense, positions and axes outside their ranges."""
import pytest
import torch

import paged_reference as R
from linear_attention_recurrence_fwd_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def case(B_, T, Hq, Hk, D, rot, dtype, A, *, cycle=False, norm=True, packed=False, seed=0, P=50):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = rnd(B_, T, (Hq + 2 * Hk) * D).to(dtype)
    q = x[..., : Hq * D].view(B_, T, Hq, D)
    k = x[..., Hq * D: (Hq + Hk) * D].view(B_, T, Hk, D)
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    c = dict(x=x, q=q, k=k, wq=None, wk=None, rope=None, axis=None, pos=None, dyq=rnd(B_, T, Hq, D).to(dtype),
             dyk=rnd(B_, T, Hk, D).to(dtype))
    if norm:
        c["wq"], c["wk"] = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)
    if rot:
        c["rope"] = B.rope_table(P, rot, device="cpu")
        share = [rot // 2 // A + (1 if a < rot // 2 % A else 0) for a in range(A)]
        c["axis"] = B.axis_map(share, cycle, device="cpu")
    c["pos"] = torch.randint(0, P, (A, B_, T), generator=g).to(torch.int32)
    return c


def up(c, packed, q):
    d = {n: (None if t is None else t.cuda()) for n, t in c.items() if n not in ("x", "q", "k")}
    Hq, D = c["q"].shape[2:]
    Hk = c["k"].shape[2]
    if packed:
        x = c["x"].cuda()
        d["q"] = x[..., : Hq * D].view(c["q"].shape)
        d["k"] = x[..., Hq * D: (Hq + Hk) * D].view(c["k"].shape)
    else:
        d["q"], d["k"] = c["q"].cuda(), c["k"].cuda()
    return d


def flat(x):
    return None if x is None else x.reshape(-1, *x.shape[2:])


def check(c, packed=False, interleaved=False, eps=1e-6, w_offset=0.0, what=""):
    d = up(c, packed, None)
    kw = dict(eps=eps, w_offset=w_offset, interleaved=interleaved)
    rot = 0 if c["rope"] is None else c["rope"].shape[1]
    tokens = c["q"].shape[0] * c["q"].shape[1]
    pos = c["pos"]
    if pos is None:
        pos = torch.arange(c["q"].shape[1]).repeat(c["q"].shape[0]).expand(4, -1)
    z = R.turns(c["rope"], c["axis"], pos.reshape(pos.shape[0], tokens)) if rot else None
    oq, ok = B.norm_rope_axes(d["q"], d["k"], d["wq"], d["wk"], d["rope"], d["axis"], d["pos"], **kw)
    g = B.norm_rope_axes_bwd(d["q"], d["k"], d["wq"], d["wk"], d["rope"], d["axis"], d["pos"], d["dyq"], d["dyk"], **kw)
    torch.cuda.synchronize()
    hs = R.half_step(c["q"].dtype)
    for n, y, dx, dw in (("q", oq, g["dq"], g["dwq"]), ("k", ok, g["dk"], g["dwk"])):
        ref, bound = R.norm_turn(flat(c[n]), c["w" + n], z, rot, interleaved, eps, w_offset)
        R.within(flat(y), ref, bound + hs * ref.abs() * 1.01, what + " " + n)
        rx, rw, bx, bw = R.norm_turn_vjp(flat(c[n]), c["w" + n], z, flat(c["dy" + n]), rot, interleaved, eps, w_offset)
        R.within(flat(dx), rx, bx + hs * rx.abs() * 1.01, what + " d" + n)
        if dw is None:
            assert rw is None
        else:
            R.within(dw, rw, bw, what + " dw" + n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("A,cycle", [(1, False), (2, True), (3, False), (3, True), (4, True)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(dtype, A, cycle, norm, interleaved):
    check(case(2, 7, 6, 2, 64, 48, dtype, A, cycle=cycle, norm=norm, seed=A), interleaved=interleaved, w_offset=0.25)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(8, 0), (16, 16), (24, 16), (40, 32), (128, 128), (136, 48), (256, 64), (512, 512), (512, 0)])
def test_head_sizes(dtype, D, rot):
    for norm in (True, False):
        check(case(3, 5, 3, 1, D, rot, dtype, 3, cycle=True, norm=norm, seed=D + rot), what="norm %d" % norm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_and_long(dtype):
    """Slices of a projection; more rows than the waves of a launch."""
    check(case(1, 300, 9, 3, 64, 64, dtype, 3, packed=True, seed=5), packed=True)
    check(case(1, 300, 9, 3, 64, 64, dtype, 3, packed=True, norm=False, seed=6), packed=True, interleaved=True)


def test_default_positions_and_axis():
    """Without positions 0 .. T-1 on every axis; without a map all pairs on the first."""
    c = case(2, 6, 2, 2, 64, 32, torch.float32, 3, seed=9)
    check(dict(c, pos=None), what="no positions")
    check(dict(c, axis=None), what="no map")
    check(dict(c, pos=None, axis=None), what="neither")


def test_outside_the_ranges():
    """A position or an axis out of range: NaN in the pairs that it concerns, and in
    the gradients of a normed row (through its mean) and of the weights."""
    c = case(1, 6, 2, 2, 64, 32, torch.float32, 3, norm=False, seed=10)
    c["pos"][0, 0, 1], c["pos"][1, 0, 2], c["pos"][2, 0, 3] = -1, 50, 2 ** 31 - 1
    c["axis"][5], c["axis"][6] = 3, 255
    check(c)
    d = up(c, False, None)
    w = torch.ones((64,), device="cuda")
    g = B.norm_rope_axes_bwd(d["q"], d["k"], w, w, d["rope"], d["axis"], d["pos"], d["dyq"], d["dyk"])
    assert torch.isnan(g["dq"]).all() and torch.isnan(g["dwq"]).sum() == 32


def test_one_axis_is_the_operator_with_one():
    """Bit for bit."""
    for dtype in (torch.bfloat16, torch.float32):
        c = up(case(2, 33, 8, 2, 128, 64, dtype, 1, seed=11), False, None)
        a = B.norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["pos"][0])
        for axis in (None, c["axis"]):
            b = B.norm_rope_axes(c["q"], c["k"], c["wq"], c["wk"], c["rope"], axis, c["pos"])
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        ga = B.norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["pos"][0], c["dyq"], c["dyk"])
        gb = B.norm_rope_axes_bwd(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["axis"], c["pos"], c["dyq"], c["dyk"])
        assert all(torch.equal(ga[n], gb[n]) for n in ga)


@pytest.mark.parametrize("norm", [True, False])
def test_autograd(norm):
    """Gradients through NormRopeAxes are the VJP's, also for cotangents that autograd
    hands on as expanded or offset views, and on a stream of their own."""
    c = up(case(2, 5, 4, 2, 64, 32, torch.float32, 3, norm=norm, seed=12), False, None)
    q, k = c["q"].requires_grad_(), c["k"].requires_grad_()
    w = [c["wq"].requires_grad_(), c["wk"].requires_grad_()] if norm else [None, None]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        oq, ok = B.NormRopeAxes.apply(q, k, *w, c["rope"], c["axis"], c["pos"])
        (oq.sum() + (torch.cat([ok.flatten(), oq.flatten()])[1:] * 2).sum()).backward()
    st.synchronize()
    dyq, dyk = torch.full_like(q, 3.0), torch.full_like(k, 2.0)
    dyk.view(-1)[0] = 0
    g = B.norm_rope_axes_bwd(q.detach(), k.detach(), *[x if x is None else x.detach() for x in w], c["rope"], c["axis"],
                             c["pos"], dyq, dyk)
    assert torch.equal(q.grad, g["dq"]) and torch.equal(k.grad, g["dk"])
    if norm:
        assert torch.equal(w[0].grad, g["dwq"]) and torch.equal(w[1].grad, g["dwk"])


@pytest.mark.parametrize("norm", [True, False])
def test_captured(norm):
    """Forward and backward replayed in a graph on new inputs."""
    c = up(case(2, 40, 4, 2, 64, 32, torch.bfloat16, 3, norm=norm, seed=13), False, None)
    args = [c[n] for n in ("q", "k", "wq", "wk", "rope", "axis", "pos")]

    def both():
        y = B.norm_rope_axes(*args)
        g = B.norm_rope_axes_bwd(*args, c["dyq"], c["dyk"])
        return [*y, *[x for x in g.values() if x is not None]]

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        both()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in range(3):
        n = case(2, 40, 4, 2, 64, 32, torch.bfloat16, 3, norm=norm, seed=20 + seed)
        for name in ("q", "k", "dyq", "dyk", "pos"):
            c[name].copy_(n[name])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, both())), seed


def test_no_tokens():
    c = up(case(2, 0, 4, 2, 64, 32, torch.bfloat16, 3, seed=14), False, None)
    oq, ok = B.norm_rope_axes(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["axis"], c["pos"])
    g = B.norm_rope_axes_bwd(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["axis"], c["pos"], c["dyq"], c["dyk"])
    assert oq.numel() == 0 and ok.numel() == 0 and not g["dwq"].any() and not g["dwk"].any()
