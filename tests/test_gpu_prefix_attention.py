"""Attention over a shared prefix and own pages against 64 bits."""
import math

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


def case(new, past, prefix, Hq, Hk, D, dtype, page, *, behind=0, by_token=False, seed=0, std=1.0, poison=True):
    """new[s] tokens behind past[s]; rows of the pool that hold nothing are NaN."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    S = len(new)
    lens = [a + b for a, b in zip(new, past)]
    counts = [-(-n // page) for n in [*lens, prefix]]
    pages = sum(counts) + 2
    order = torch.randperm(pages, generator=g)
    k, v = (rnd(pages, Hk, page, D).to(dtype) for _ in range(2))
    table = torch.full((S, max(1, max(counts[:S]))), -7, dtype=torch.int32)
    held = torch.zeros((pages, page), dtype=torch.bool)
    at = 0
    for s, n in enumerate(counts):
        ids = order[at: at + n]
        at += n
        if s < S:
            table[s, :n] = ids
        L = lens[s] if s < S else prefix
        for j, p in enumerate(ids):
            held[p, : max(0, min(page, L - j * page))] = True
    prefix_pages = ids.to(torch.int32) if prefix else None
    if poison:
        k.masked_fill_(~held[:, None, :, None], math.nan)
        v.masked_fill_(~held[:, None, :, None], math.nan)
    return dict(q=(std * rnd(sum(new) + behind, Hq, D)).to(dtype), k=k, v=v, table=table, by_token=by_token,
                lens=torch.tensor(lens, dtype=torch.int32), prefix_pages=prefix_pages, prefix=prefix,
                cu=torch.tensor([0, *new]).cumsum(0).to(torch.int32))


def up(c):
    d = {n: None if c[n] is None else c[n].cuda() for n in ("q", "k", "v", "table", "lens", "prefix_pages", "cu")}
    if c["by_token"]:
        for n in ("k", "v"):
            d[n] = d[n].transpose(1, 2).contiguous().transpose(1, 2)
    return d


def run(c, d=None, uniform=False, **kw):
    d = d or up(c)
    return B.prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["prefix_pages"], c["prefix"],
                              None if uniform else d["cu"], lse=True, **kw)


def check(c, uniform=False, scale=None, max_q=None, max_len=None, what=""):
    d = up(c)
    out = torch.full_like(d["q"], 5.0)
    o, lse = run(c, d, uniform, scale=scale, max_q=max_q, max_len=max_len, out=out)
    torch.cuda.synchronize()
    assert o is out
    D = c["q"].shape[2]
    ref = R.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["prefix_pages"], c["prefix"],
                      None if uniform else c["cu"], D ** -0.5 if scale is None else scale, max_q, max_len)
    end = c["q"].shape[0] if uniform else int(c["cu"][-1])
    R.within(o[:end], ref[0][:end], ref[2][:end], what + " o")
    R.within(lse[:end], ref[1][:end], ref[3][:end], what + " lse")
    assert (o[end:] == 5).all()
    return o


BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@BOTH
@pytest.mark.parametrize("D", [8, 40, 64, 72, 128, 136, 192, 200, 256])
def test_head_sizes(dtype, D):
    check(case([1, 3, 2], [5, 0, 40], 37, 4, 2, D, dtype, 16, seed=D))


@BOTH
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("by_token", [False, True])
def test_pages(dtype, page, by_token):
    """Pages smaller and larger than a tile, ends inside both, NaN behind the ends."""
    check(case([1, 1, 1, 1], [0, 15, 16, 130], 77, 6, 2, 64, dtype, page, by_token=by_token, seed=page), uniform=True)


@BOTH
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 600])
def test_prefix_lengths(dtype, prefix):
    check(case([1, 2, 1], [3, 0, 20], prefix, 4, 1, 64, dtype, 16, seed=prefix))


@BOTH
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (7, 1), (8, 1), (16, 1), (17, 1), (32, 1), (40, 1), (24, 3)])
def test_heads(dtype, heads):
    check(case([1, 2], [30, 7], 70, *heads, 64, dtype, 16, seed=heads[0]))


@BOTH
@pytest.mark.parametrize("new", [[1], [2, 2], [5, 0, 1, 33], [70], [0, 0, 9], [1] * 40])
@pytest.mark.parametrize("prefix", [0, 90])
def test_ragged(dtype, new, prefix):
    """Empty sequences, rows behind the last, one token to several tiles of rows."""
    past = [(7 * s) % 50 for s in range(len(new))]
    check(case(new, past, prefix, 4, 2, 64, dtype, 8, behind=3, seed=len(new)))


@BOTH
def test_long_own_keys(dtype):
    """Own keys over many splits, of very unequal lengths."""
    check(case([1, 1, 2, 1], [1500, 0, 700, 255], 300, 4, 2, 64, dtype, 32, seed=1))
    check(case([1, 1, 2, 1], [1500, 0, 700, 255], 0, 4, 2, 64, dtype, 32, seed=2))


def test_many_rows():
    """More rows of the prefix than one item takes, by wide heads."""
    check(case([1] * 30, [3 * s for s in range(30)], 200, 16, 2, 128, torch.bfloat16, 16, seed=3), uniform=True)
    check(case([20, 31], [0, 11], 150, 8, 1, 256, torch.bfloat16, 16, seed=4))


@BOTH
def test_no_key_at_all(dtype):
    """lens smaller than the call's tokens: the first of them see nothing: zeros, and
    the prefix alone where there is one."""
    for prefix in (0, 20):
        c = case([4, 2], [0, 6], prefix, 2, 1, 64, dtype, 8, seed=5)
        c["lens"][0] = 2
        o = check(c)
        if not prefix:
            assert not o[:2].any()
        c["lens"][0] = 0
        check(c)


@BOTH
def test_large_scores(dtype):
    """Scores of several hundred, growing and falling along the keys, and a scale of its own."""
    c = case([1, 2], [200, 90], 150, 2, 1, 64, dtype, 16, seed=6, poison=False)
    up_, down = torch.linspace(-4, 4, 16), torch.linspace(4, -4, 16)
    c["k"][::2] *= up_[None, None, :, None].to(dtype)
    c["k"][1::2] *= down[None, None, :, None].to(dtype)
    check(c, scale=3.0)
    check(c, scale=-0.5)
    check(c, scale=0.0)


@BOTH
def test_infinities_and_nan_in_keys(dtype):
    """NaN in a key that a token sees reaches that token; those before it do not see it."""
    c = case([3], [5], 0, 2, 1, 64, dtype, 8, seed=7)
    p = int(c["table"][0, 0])
    c["k"][p, 0, 6] = math.nan   # the call's second token
    o = check(c)
    assert torch.isfinite(o[0].float()).all() and torch.isnan(o[1:].float()).all()
    c = case([1, 1], [5, 5], 9, 2, 1, 64, dtype, 8, seed=8)
    c["v"][int(c["table"][0, 0]), 0, 2, 3] = math.inf
    c["v"][int(c["prefix_pages"][0]), 0, 2, 5] = -math.inf
    check(c)


@BOTH
def test_pages_that_do_not_exist(dtype):
    """Rows of NaN for those who see them, nobody else."""
    c = case([1, 1, 1], [20, 20, 3], 0, 2, 1, 64, dtype, 8, seed=9)
    c["table"][0, 1] = c["k"].shape[0]
    c["table"][1, 2] = -1
    o = check(c)
    assert torch.isnan(o[:2].float()).all() and torch.isfinite(o[2].float()).all()
    c = case([1, 1], [20, 3], 30, 2, 1, 64, dtype, 8, seed=10)
    c["prefix_pages"][2] = 2 ** 31 - 1
    assert torch.isnan(check(c).float()).all()


@BOTH
@pytest.mark.parametrize("prefix", [0, 40, 300])
def test_lengths_out_of_bounds(dtype, prefix):
    """More tokens than max_q, or own keys outside 0 .. max_len: NaN for that sequence."""
    c = case([2, 5, 40, 1], [3, 10, 60, 2], prefix, 4, 2, 64, dtype, 8, seed=11)
    check(c, max_q=5)
    check(c, max_q=1)
    check(c, max_len=15)
    check(c, max_len=0)
    c["lens"][0], c["lens"][3] = -1, 2 ** 31 - 1
    check(c, max_q=40, max_len=104)


@BOTH
def test_many_sequences(dtype):
    """Enough sequences for one item to go through prefix and own keys together."""
    new = [1 + (s * 7) % 3 for s in range(300)]
    past = [(s * 11) % 40 for s in range(300)]
    check(case(new, past, 50, 4, 2, 64, dtype, 16, behind=2, seed=12), max_q=3)
    check(case([1] * 300, past, 50, 4, 2, 64, dtype, 16, seed=13), uniform=True)


def test_far_pages():
    """A pool of more than 4 GiB and 2^31 elements."""
    pages, Hk, page, D = 34000, 2, 128, 256
    k = torch.empty((pages, Hk, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((pages, Hk, page, D), dtype=torch.bfloat16, device="cuda")
    c = case([1, 1], [200, 100], 140, 4, Hk, D, torch.bfloat16, page, seed=14, poison=False)
    far = torch.tensor([pages - 1, 0, 33000, 16384, pages - 2, 7, 32768, 1][: c["k"].shape[0]])
    for i, p in enumerate(far):
        k[p], v[p] = c["k"][i].cuda(), c["v"][i].cuda()
    d = up(c)
    move = lambda t: far.to(torch.int32)[t.clamp(min=0).long()].cuda()  # noqa: E731
    d.update(k=k, v=v, table=move(c["table"]), prefix_pages=move(c["prefix_pages"]))
    a, b = run(c, uniform=True), run(c, d, uniform=True)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@BOTH
def test_same_bits(dtype):
    """Twice, on another stream, two at once on two streams, and replayed on other
    inputs: the same bits."""
    c = case([1, 4, 2], [300, 5, 90], 260, 4, 2, 64, dtype, 16, seed=15)
    e = case([1, 4, 2], [300, 5, 90], 260, 4, 2, 64, dtype, 16, seed=16)
    d, f = up(c), up(e)
    a, b = run(c, d, max_q=4), run(e, f, max_q=4)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        with torch.cuda.stream(st[0]):
            a2 = run(c, d, max_q=4)
        with torch.cuda.stream(st[1]):
            b2 = run(e, f, max_q=4)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([*a, *b], [*a2, *b2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = run(c, d, max_q=4)
    old = {n: d[n].clone() for n in ("q", "k", "v", "table", "lens", "prefix_pages", "cu")}
    for src, ref in ((f, b), (old, a), (f, b)):
        for n in old:
            d[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(g, ref))


def test_no_tokens():
    c = case([0, 0], [3, 0], 5, 2, 1, 64, torch.bfloat16, 8, seed=17)
    o, lse = run(c)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)


def test_append_then_attend():
    """A batch of two prompts behind a shared prefix, then single tokens, as a program
    serves them: the prefix and every token appended with norm and rotation, attention
    over what the cache holds, against attention over all keys at once in 64 bits."""
    g = torch.Generator().manual_seed(18)
    Hq, Hk, D, rot, page, prefix = 4, 2, 64, 32, 16, 45
    w = [(1 + 0.1 * torch.randn(D, generator=g)) for _ in range(2)]
    rope = B.rope_table(200, rot, device="cpu")
    kp = torch.full((40, Hk, page, D), math.nan, dtype=torch.float32, device="cuda")
    vp = torch.full_like(kp, math.nan)
    dev = dict(wq=w[0].cuda(), wk=w[1].cuda(), rope=rope.cuda())
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    shared = i32(31, 2, 17)
    table = i32([5, 9, 33], [12, 30, 1])
    rows = lambda n: torch.randn((n, Hq + 2 * Hk, D), generator=g)  # noqa: E731
    x = rows(prefix)
    B.paged_append(x[:, :Hq].cuda(), x[:, Hq: Hq + Hk].cuda(), x[:, Hq + Hk:].cuda(), kp, vp, shared.view(1, 3), i32(0), **dev)
    seen = [[x], [x]]  # per sequence all tokens so far
    past = [0, 0]
    for new in ([7, 12], [1, 1], [1, 1], [3, 0], [1, 1]):
        x = rows(sum(new))
        cu = i32(0, new[0], sum(new))
        q = B.paged_append(x[:, :Hq].cuda(), x[:, Hq: Hq + Hk].cuda(), x[:, Hq + Hk:].cuda(), kp, vp, table, i32(*past), cu,
                           first=prefix, **dev)
        past = [a + b for a, b in zip(past, new)]
        o = B.prefix_attention(q, kp, vp, table, i32(*past), shared, prefix, cu, max_q=max(new))
        torch.cuda.synchronize()
        at = 0
        for s, n in enumerate(new):
            seen[s].append(x[at: at + n])
            every = torch.cat(seen[s])
            z = R.turns(rope, None, torch.arange(every.shape[0])[None])
            qq, _ = R.norm_turn(every[:, :Hq], w[0], z, rot, False, 1e-6, 0.0)
            kk, _ = R.norm_turn(every[:, Hq: Hq + Hk], w[1], z, rot, False, 1e-6, 0.0)
            vv = every[:, Hq + Hk:].double()
            T = every.shape[0]
            for h in range(Hq):
                a = qq[T - n:, h] @ kk[:, h // 2].T * D ** -0.5
                a.masked_fill_(torch.arange(T)[None] > torch.arange(T - n, T)[:, None], -math.inf)
                ref = torch.softmax(a, -1) @ vv[:, h // 2]
                # keys and queries are off by (D/16 + 12) half steps, the scores by
                # twice that and the product's (D + 4); see attention()'s bound
                d = (2 * (D / 16 + 12) + D + 4) * R.U32 * D ** -0.5 * (qq[T - n:, h].abs() @ kk[:, h // 2].abs().T).max() if n else 0
                bound = (2 * d + (T / 8 + 66) * R.U32) * vv.abs().max()
                assert n == 0 or (o[at: at + n, h].double().cpu() - ref).abs().max() <= bound
            at += n
