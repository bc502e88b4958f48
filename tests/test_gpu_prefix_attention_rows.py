"""A row's bits are its own: what lies beside it in its tile of rows does not reach them,
not even where its weights' sum lies on the bound that moves the softmax's reference."""
import math

import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def sums(order):
    """A lane's sixteen weights as a block adds them, in a tree, and one after the other, in fp32."""
    x = torch.tensor(order, dtype=torch.float32)
    t = x
    while t.numel() > 1:
        t = t[0::2] + t[1::2]
    s = torch.zeros((), dtype=torch.float32)
    for y in x:
        s = s + y
    return float(t), float(s)


def test_a_sum_on_the_bound():
    """Sixteen weights relative to the reference, of one lane: 2^16 in the last place and
    2^-9 in four others, so that their sum is 2^16 in the tree's order, the bound, and above
    it in turn.  The rows' scores come from two channels; a row beside them (its own channel)
    exceeds the bound in that very block."""
    D, n, rows = 64, 96, 40
    order = [-200.0] * 16
    order[15] = 16.0
    for i in (0, 8, 12, 14):
        order[i] = -9.0
    tree, turn = sums([2.0 ** x for x in order])
    assert tree == 65536 < turn
    g = torch.Generator().manual_seed(0)
    score = torch.full((n,), -200.0)
    score[:32] = -(1 + torch.randint(0, 640, (32,), generator=g) / 128.0)  # (two bf16 channels of them below)
    score[5] = 0.0                                                         # the first block's maximum: the reference
    for i in range(16):                                                    # the second block, half of the lanes
        score[32 + 8 * (i // 4) + i % 4] = order[i]
    score[64:] = -(torch.randint(0, 1024, (32,), generator=g) / 128.0)
    whole = score.round()
    k = torch.zeros((n // 16, 1, 16, D), dtype=torch.bfloat16)
    flat = k.view(n, D)
    flat[:, 0], flat[:, 1] = whole.bfloat16(), (score - whole).bfloat16()
    assert torch.equal(flat[:, 0].float() + flat[:, 1].float(), score)
    flat[32:64, 2] = 40.0                                                  # seen by the rows beside alone
    v = torch.randn((n // 16, 1, 16, D), generator=g).bfloat16()
    q = torch.zeros((rows, 4, D), dtype=torch.bfloat16)
    q[:, :, 0] = q[:, :, 1] = 1
    beside = q.clone()
    beside[::3, 1, 2] = 1
    own = torch.zeros((1, 1, 16, D), dtype=torch.bfloat16)
    pool_k, pool_v = torch.cat([k, own]).cuda(), torch.cat([v, own]).cuda()
    prefix = torch.arange(n // 16, dtype=torch.int32, device="cuda")
    table = torch.full((rows, 1), n // 16, dtype=torch.int32, device="cuda")
    lens = torch.ones(rows, dtype=torch.int32, device="cuda")
    run = lambda x: B.prefix_attention(x.cuda(), pool_k, pool_v, table, lens, prefix, n, scale=math.log(2), lse=True)  # noqa: E731
    (a, la), (b, lb) = run(q), run(beside)
    torch.cuda.synchronize()
    same = torch.ones((rows, 4), dtype=torch.bool)
    same[::3, 1] = False
    assert not torch.equal(lb[~same], la[~same])
    assert torch.equal(a[same], b[same]) and torch.equal(la[same], lb[same])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 256])
def test_rows_behind_the_last_sequence(dtype, D):
    """A padded batch: whatever the queries behind cu[S] hold, NaN or infinities among it, the
    others' results have the same bits and the rows behind stay as they were."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    new, pad, prefix = [30, 0, 25, 1], 40, 700
    lens = torch.tensor([33, 4, 60, 16], dtype=torch.int32, device="cuda")
    k, v = rnd(44 + 16, 2, 16, D), rnd(44 + 16, 2, 16, D)
    pages = torch.arange(44, dtype=torch.int32, device="cuda")
    table = torch.arange(44, 60, dtype=torch.int32, device="cuda").view(4, 4)
    cu = torch.tensor([0, *new], device="cuda").cumsum(0).to(torch.int32)
    end = sum(new)
    q = rnd(end + pad, 8, D)
    ref = B.prefix_attention(q[:end].contiguous(), k, v, table, lens, pages, prefix, cu, max_q=30, lse=True)
    first = None
    for fill in (None, math.nan, math.inf, -math.inf, 1e30):
        x = q.clone()
        if fill is not None:
            x[end:] = fill
        out = torch.full_like(x, 5.0)
        o, lse = B.prefix_attention(x, k, v, table, lens, pages, prefix, cu, max_q=30, lse=True, out=out)
        torch.cuda.synchronize()
        assert o is out and (o[end:] == 5).all()
        first = (o[:end].clone(), lse[:end].clone()) if first is None else first
        assert torch.equal(o[:end], first[0]) and torch.equal(lse[:end], first[1])
    # (other tiles of rows and splits: the same up to roundings)
    close = 2 ** -7 if dtype == torch.bfloat16 else 1e-5
    assert (first[0].double() - ref[0].double()).abs().max() <= close * v.double().abs().max()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 330])
def test_rows_of_nan_among_others(D, prefix):
    """Queries of NaN in every wave of a causal prompt, whose first rows see few keys or (a
    length smaller than the call's tokens) none: NaN there, the others' bits as without them."""
    g = torch.Generator(device="cuda").manual_seed(D)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    new, lens = [150, 90], [120, 400]
    pages = -(-prefix // 16)
    k, v = rnd(pages + 60, 2, 16, D), rnd(pages + 60, 2, 16, D)
    shared = torch.arange(pages, dtype=torch.int32, device="cuda") if prefix else None
    table = torch.arange(pages, pages + 60, dtype=torch.int32, device="cuda").view(2, 30)
    cu = torch.tensor([0, *new], device="cuda").cumsum(0).to(torch.int32)
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = 3 * rnd(sum(new), 4, D)
    x = q.clone()
    x[5::13, 1, 7] = math.nan
    (a, la), (b, lb) = (B.prefix_attention(y, k, v, table, length, shared, prefix, cu, max_q=150, lse=True) for y in (q, x))
    torch.cuda.synchronize()
    bad = torch.isnan(x.float()).any(-1)
    if not prefix:
        bad[:30] = False  # (no key at all: zeros, whatever the query)
        assert not b[:30].any() and (lb[:30] == -math.inf).all()
    assert torch.isnan(b[bad].float()).all() and torch.isnan(lb[bad]).all()
    assert torch.equal(a[~bad], b[~bad]) and torch.equal(la[~bad], lb[~bad])
