"""Attention over pages where a launch is large: a ragged batch of many sequences whose
longest is not named, and few key heads with one split of the prefix."""
import pytest
import torch

import paged_reference as R
from linear_attention_recurrence_fwd_amd import binding as B
from test_gpu_prefix_attention import case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


@pytest.mark.parametrize("prefix", [0, 40])
def test_a_ragged_batch_without_its_longest(prefix):
    """16384 tokens of 512 sequences, 32 heads on 8: as with max_q given, and some of its
    sequences against 64 bits."""
    g = torch.Generator().manual_seed(1)
    S, Hq, Hk, D, page = 512, 32, 8, 64, 16
    new = torch.randint(0, 64, (S,), generator=g)
    new[-1] += 16384 - new.sum() if new.sum() < 16384 else 0
    while new.sum() > 16384:
        new[int(new.argmax())] -= 1
    N, width = int(new.sum()), -(-int(new.max()) // page) + 1
    past = torch.randint(0, page, (S,), generator=g)
    k, v = (torch.randn((3 + S * width, Hk, page, D), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((N, Hq, D), generator=g).bfloat16()
    table = (3 + torch.randperm(S * width, generator=g).view(S, width)).to(torch.int32)
    lens, shared = (new + past).to(torch.int32), torch.tensor([2, 0, 1], dtype=torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32)
    d = [x.cuda() for x in (q, k, v, table, lens)]
    pages = shared.cuda() if prefix else None
    a, la = B.prefix_attention(*d, pages, prefix, cu.cuda(), lse=True)
    b, lb = B.prefix_attention(*d, pages, prefix, cu.cuda(), max_q=int(new.max()), lse=True)
    torch.cuda.synchronize()
    assert N == 16384 and torch.isfinite(a.float()).all()
    # the tiles of rows are the same, the splits of keys need not be: two roundings
    assert (a.double() - b.double()).abs().max() <= 2 * 2 ** -8 * v.double().abs().max()
    assert (la - lb).abs().max() <= 1e-5 * la.abs().max()
    for s in (0, 255, S - 1):
        t0, t1 = int(cu[s]), min(int(cu[s + 1]), int(cu[s]) + 8)
        if t1 == t0:
            continue
        some = torch.tensor([0, t1 - t0], dtype=torch.int32)
        length = (past[s: s + 1] + (t1 - t0)).to(torch.int32)
        ref = R.attention(q[t0:t1], k, v, table[s: s + 1], length, shared, prefix, some, D ** -0.5)
        R.within(a[t0:t1], ref[0], ref[2], "o of sequence %d" % s)
        R.within(la[t0:t1], ref[1], ref[3], "lse of sequence %d" % s)


def test_refusal_names_max_q():
    """A ragged batch that no launch holds as long as max_q is the whole of it; with its
    longest sequence's tokens it runs."""
    N, S, Hq, Hk, D = 1 << 16, 1 << 12, 32, 8, 8
    z = torch.zeros
    q = z((N, Hq, D), dtype=torch.bfloat16, device="cuda")
    kp = z((4, Hk, 16, D), dtype=torch.bfloat16, device="cuda")
    table, lens = z((S, 1), dtype=torch.int32, device="cuda"), torch.full((S,), 16, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, N + 1, N // S, dtype=torch.int32, device="cuda")
    with pytest.raises(B.GdnError, match="UNSUPPORTED.*max_q = 65536 .*4096 sequences") as e:
        B.prefix_attention(q, kp, kp.clone(), table, lens, cu=cu)
    assert e.value.code == 2
    assert not B.prefix_attention(q, kp, kp.clone(), table, lens, cu=cu, max_q=16).any()


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (6, 3), (14, 7), (9, 9), (20, 10)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tiles_by_few_heads(dtype, heads):
    """Numbers of splits by key heads below, at and above eight, by several tiles of rows."""
    check(case([40, 1, 33], [4, 0, 20], 70, *heads, 64, dtype, 16, seed=heads[0]))
