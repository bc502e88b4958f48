"""Appending to a paged cache against 64 bits: turned queries, the written rows, and
everything else in the pool as it was."""
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


def case(new, past, Hq, Hk, D, rot, dtype, page, *, A=0, norm=True, behind=0, by_token=False, seed=0, P=200, spare=2):
    """new[s] tokens behind past[s]; `behind` rows behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    N, S = sum(new) + behind, len(new)
    counts = [-(-(a + b) // page) for a, b in zip(new, past)]
    order = torch.randperm(sum(counts) + spare, generator=g)
    table = torch.full((S, max(1, max(counts))), -7, dtype=torch.int32)
    at = 0
    for s, n in enumerate(counts):
        table[s, :n] = order[at: at + n]
        at += n
    x = rnd(N, (Hq + 2 * Hk) * D).to(dtype)
    shape = (sum(counts) + spare, Hk, page, D)
    pools = [rnd(*shape).to(dtype) for _ in range(2)]
    return dict(x=x, H=(Hq, Hk, D), k_pages=pools[0], v_pages=pools[1], table=table, by_token=by_token,
                past=torch.tensor(past, dtype=torch.int32),
                cu=torch.tensor([0, *new]).cumsum(0).to(torch.int32),
                wq=1 + 0.1 * rnd(D) if norm else None, wk=1 + 0.1 * rnd(D) if norm else None,
                rope=B.rope_table(P, rot, device="cpu") if rot else None,
                axis=B.axis_map([rot // 2 // A + (a < rot // 2 % A) for a in range(A)], True, device="cpu") if A and rot else None,
                pos=torch.randint(0, P, (A, N), generator=g).to(torch.int32) if A else None)


def split(x, H):
    Hq, Hk, D = H
    x = x.unflatten(-1, (Hq + 2 * Hk, D))
    return x[:, :Hq], x[:, Hq: Hq + Hk], x[:, Hq + Hk:]


def pool(x, by_token):
    x = x.cuda()
    return x.transpose(1, 2).contiguous().transpose(1, 2) if by_token else x


def run(c, uniform=False, packed=True, queries=True, first=0, interleaved=False, w_offset=0.0, eps=1e-6, out=None):
    q, k, v = split(c["x"].cuda(), c["H"])
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    d = {n: None if c[n] is None else c[n].cuda() for n in ("table", "past", "cu", "wq", "wk", "rope", "axis", "pos")}
    kp, vp = pool(c["k_pages"], c["by_token"]), pool(c["v_pages"], c["by_token"])
    oq = B.paged_append(q if queries else None, k, v, kp, vp, d["table"], d["past"], None if uniform else d["cu"],
                        wq=d["wq"] if queries else None, wk=d["wk"], rope=d["rope"], axis=d["axis"], pos=d["pos"],
                        first=first, eps=eps, w_offset=w_offset, interleaved=interleaved, out=out)
    torch.cuda.synchronize()
    return oq, kp, vp


def check(c, uniform=False, first=0, queries=True, **kw):
    N = c["x"].shape[0]
    out = torch.full((N, c["H"][0], c["H"][2]), 5.0, dtype=c["x"].dtype, device="cuda") if queries else None
    oq, kp, vp = run(c, uniform, first=first, queries=queries, out=out, **kw)
    eps, w_offset, inter = kw.get("eps", 1e-6), kw.get("w_offset", 0.0), kw.get("interleaved", False)
    rot = 0 if c["rope"] is None else c["rope"].shape[1]
    cu = None if uniform else c["cu"]
    where = R.places(c["past"], cu, len(c["past"]), N)
    pos = c["pos"]
    if pos is None:
        pos = torch.tensor([0 if s is None else first + at for s, _, at in where]).expand(4, -1)
    z = R.turns(c["rope"], c["axis"], pos) if rot else None
    q, k, v = split(c["x"], c["H"])
    hs = R.half_step(c["x"].dtype)
    live = torch.tensor([s is not None for s, _, _ in where])
    if queries:
        ref, bound = R.norm_turn(q, c["wq"], z, rot, inter, eps, w_offset)
        R.within(oq[live.cuda()], ref[live], (bound + hs * ref.abs() * 1.01)[live], "queries")
        assert (oq[~live.cuda()] == 5).all()
    ref, bound = R.norm_turn(k, c["wk"], z, rot, inter, eps, w_offset)
    rk, rv, put = R.append(ref, v, c["k_pages"], c["v_pages"], c["table"], c["past"], cu)
    bk, _, _ = R.append(bound + hs * ref.abs() * 1.01, v, torch.zeros_like(rk), torch.zeros_like(rk), c["table"], c["past"], cu)
    R.within(kp, rk, bk, "keys")  # (a bound of 0 where nothing was written)
    assert torch.equal(vp.double().cpu(), rv)
    return put


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [1, 4, 16, 64])
@pytest.mark.parametrize("by_token", [False, True])
def test_ragged(dtype, page, by_token):
    """Empty sequences among others, pages that end inside a prompt, rows behind the last."""
    c = case([3, 0, 17, 1, 0], [5, 9, 0, 63, 0], 6, 2, 64, 32, dtype, page, A=3, behind=4, by_token=by_token, seed=page)
    assert check(c).sum() == 21


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(8, 0), (16, 16), (24, 16), (72, 32), (128, 128), (200, 48), (256, 64), (256, 256)])
@pytest.mark.parametrize("norm", [True, False])
def test_head_sizes(dtype, D, rot, norm):
    check(case([2, 5], [3, 0], 5, 1, D, rot, dtype, 8, norm=norm, seed=D), first=7, interleaved=norm, w_offset=0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_single_tokens(dtype):
    """One token each, with and without offsets; dense rows; keys and values alone."""
    c = case([1] * 9, [0, 1, 2, 15, 16, 17, 31, 32, 100], 8, 2, 128, 64, dtype, 16, seed=3)
    check(c, uniform=True)
    check(c, packed=False)
    check(c, uniform=True, queries=False)
    check(dict(c, wq=None, wk=None), uniform=True, queries=False, first=20)


def test_several_tokens_each():
    check(case([4] * 7, [1, 2, 3, 4, 5, 6, 7], 4, 4, 64, 64, torch.bfloat16, 4, seed=4), uniform=True)


def test_many_sequences():
    """More sequences than one look-up of sixty-four."""
    g = torch.Generator().manual_seed(1)
    new = torch.randint(0, 3, (700,), generator=g).tolist()
    past = torch.randint(0, 40, (700,), generator=g).tolist()
    check(case(new, past, 2, 1, 64, 32, torch.bfloat16, 16, seed=5, behind=3))
    new = [0] * 4200
    new[4100], new[63], new[64] = 2, 1, 3
    check(case(new, [1] * 4200, 2, 1, 16, 16, torch.float32, 4, seed=6))


def test_places_that_do_not_exist():
    """Behind the table's row, before its begin, on pages outside the pool: nothing is
    written there, the queries are."""
    c = case([3, 3, 3, 3], [2, 6, 0, 1], 2, 1, 64, 32, torch.float32, 4, seed=7)
    c["past"][1] = 7      # the last two of three behind the row's room (3 pages of 4)
    c["past"][2] = -2     # the first two before the begin
    c["table"][0, 1] = c["k_pages"].shape[0]
    c["table"][3, 0] = -1
    c["table"] = c["table"][:, :2].contiguous()
    put = check(c, first=10)
    assert put.sum() == 2 + 1 + 1 + 0 or put.sum() >= 3
    c["past"][1] = 2 ** 31 - 1
    check(dict(c, pos=torch.zeros((1, 12), dtype=torch.int32)))


def test_positions_outside_the_table():
    """NaN in the turned channels, written like any other."""
    check(case([2, 2], [198, 0], 2, 1, 64, 32, torch.float32, 8, norm=False, seed=8), first=1)


def test_keys_beside_values():
    """Keys and values in one tensor [pages, 2, Hk, page, D]."""
    c = case([5, 3], [2, 9], 2, 2, 64, 32, torch.bfloat16, 4, seed=9)
    both = torch.stack([c["k_pages"], c["v_pages"]], 1).cuda()
    oq, kp, vp = run(c)
    q, k, v = split(c["x"].cuda(), c["H"])
    d = {n: c[n].cuda() for n in ("table", "past", "cu", "wq", "wk", "rope")}
    o2 = B.paged_append(q, k, v, both[:, 0], both[:, 1], d["table"], d["past"], d["cu"], wq=d["wq"], wk=d["wk"], rope=d["rope"])
    torch.cuda.synchronize()
    assert torch.equal(oq, o2) and torch.equal(both[:, 0], kp) and torch.equal(both[:, 1], vp)


def test_far_pages():
    """A pool of more than 4 GiB and 2^31 elements: pages at both ends."""
    pages, Hk, page, D = 34000, 2, 128, 256
    kp = torch.empty((pages, Hk, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty((pages, Hk, page, D), dtype=torch.bfloat16, device="cuda")
    ids = [pages - 1, 0, 32768, pages - 2]
    for i in ids:
        kp[i], vp[i] = 1.0, 2.0
    x = torch.randn((4, 2 * Hk, D), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    table = torch.tensor(ids, dtype=torch.int32, device="cuda").view(4, 1)
    past = torch.tensor([127, 0, 64, 5], dtype=torch.int32, device="cuda")
    assert B.paged_append(None, x[:, :Hk], x[:, Hk:], kp, vp, table, past) is None
    torch.cuda.synchronize()
    for s, i in enumerate(ids):
        rk, rv = torch.full_like(kp[i], 1.0), torch.full_like(vp[i], 2.0)
        rk[:, int(past[s])], rv[:, int(past[s])] = x[s, :Hk], x[s, Hk:]
        assert torch.equal(kp[i], rk) and torch.equal(vp[i], rv)


def test_captured_and_other_stream():
    c = case([1] * 5, [3, 4, 5, 6, 7], 4, 2, 64, 32, torch.bfloat16, 8, seed=10)
    q, k, v = split(c["x"].cuda(), c["H"])
    d = {n: c[n].cuda() for n in ("table", "past", "wq", "wk", "rope", "k_pages", "v_pages")}
    kw = dict(wq=d["wq"], wk=d["wk"], rope=d["rope"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        B.paged_append(q, k, v, d["k_pages"], d["v_pages"], d["table"], d["past"], **kw)
    torch.cuda.current_stream().wait_stream(st)
    ref = run(c, uniform=True)
    torch.cuda.synchronize()
    assert torch.equal(d["k_pages"], ref[1]) and torch.equal(d["v_pages"], ref[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oq = B.paged_append(q, k, v, d["k_pages"], d["v_pages"], d["table"], d["past"], **kw)
    for past in ([0, 0, 0, 0, 0], [4, 3, 2, 1, 0], [8, 9, 10, 0, 1]):
        c["past"] = torch.tensor(past, dtype=torch.int32)
        d["past"].copy_(c["past"])
        for n in ("k_pages", "v_pages"):
            d[n].copy_(c[n])
        graph.replay()
        torch.cuda.synchronize()
        ref = run(c, uniform=True)
        assert torch.equal(oq, ref[0]) and torch.equal(d["k_pages"], ref[1]) and torch.equal(d["v_pages"], ref[2])


def test_no_tokens():
    c = case([0, 0], [3, 0], 2, 1, 64, 32, torch.bfloat16, 8, seed=11)
    oq, kp, vp = run(c)
    assert oq.shape == (0, 2, 64) and torch.equal(kp.cpu(), c["k_pages"]) and torch.equal(vp.cpu(), c["v_pages"])
