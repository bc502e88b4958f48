"""Attention over a shared prefix and own pages with many rows (bf16, more than 64 rows
of a key head's queries), against 64 bits."""
import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B
from test_gpu_prefix_attention import case, check, run, up

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


@pytest.mark.parametrize("prefix", [0, 203])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 104, 128, 136, 192, 200, 248, 256])
def test_head_sizes(D, prefix):
    """Heads of every class of the kernel, whole and not, by prompts with a causal end."""
    check(case([45, 3, 70], [5, 0, 90], prefix, 4, 2, D, BF16, 16, seed=D))


@pytest.mark.parametrize("D", [64, 136, 256])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 64, 256])
@pytest.mark.parametrize("by_token", [False, True])
def test_pages(D, page, by_token):
    """Pages smaller and larger than a wave's rows of a tile, ends inside both."""
    check(case([33, 1, 20], [0, 130, 31], 77, 6, 2, D, BF16, page, by_token=by_token, seed=page))


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("prefix", [1, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 600])
def test_prefix_lengths(D, prefix):
    check(case([1] * 17, [s % 5 for s in range(17)], prefix, 8, 1, D, BF16, 16, seed=prefix), uniform=True)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("new", [[65], [64, 1], [127], [128], [129], [257], [0, 66, 0, 31], [16] * 9])
def test_row_tiles(D, new):
    """Tiles of rows that end anywhere, with own keys before the call's and none."""
    for past in (0, 37):
        check(case(new, [past * (s % 2) for s in range(len(new))], 90, 2, 1, D, BF16, 32, behind=3, seed=len(new) + past))


@pytest.mark.parametrize("heads", [(1, 1), (3, 1), (7, 1), (12, 4), (40, 1)])
def test_heads(heads):
    """Numbers of query heads to a key head that divide no tile."""
    check(case([70, 22], [3, 50], 100, *heads, 64, BF16, 16, seed=heads[0]))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_reference_moves(D):
    """Scores that grow along the keys by hundreds, in the prefix and in the own keys, for
    some rows and not for others: the reference is moved in every block, of a tile's
    blocks in the first, the second and both."""
    c = case([40, 30], [300, 10], 500, 4, 2, D, BF16, 16, seed=D)
    k = c["k"]
    for ids, n in ((c["prefix_pages"], 500), (c["table"][0], 340), (c["table"][1], 40)):
        for j in range(0, n, 16):
            k[int(ids[j // 16])] *= 0.02 * j
    c["q"][::3] *= 0.01
    check(c, scale=1.0)
    check(c, scale=-1.0)
    c["q"][:, :, : D // 2] = 0
    check(c, scale=0.3)


@pytest.mark.parametrize("D", [72, 256])
def test_rows_without_keys(D):
    """Rows that see nothing of their own among rows that do, without a prefix and with one."""
    for prefix in (0, 50):
        c = case([80, 70], [0, 6], prefix, 2, 1, D, BF16, 8, seed=5)
        c["lens"][0] = 33  # its first 47 tokens see none
        o = check(c)
        if not prefix:
            assert not o[:47].any()


@pytest.mark.parametrize("D", [64, 200])
def test_pages_and_lengths_that_do_not_exist(D):
    c = case([70, 68, 3], [20, 20, 3], 0, 2, 1, D, BF16, 8, seed=9)
    c["table"][0, 1] = c["k"].shape[0]
    c["table"][1, 2] = -1
    o = check(c)
    assert torch.isfinite(o[138:].float()).all()
    c = case([70, 3, 66], [20, 4, 3], 40, 2, 1, D, BF16, 8, seed=10)
    check(c, max_q=69)
    check(c, max_len=80)
    c["prefix_pages"][2] = 2 ** 31 - 1
    assert torch.isnan(check(c).float()).all()


def test_a_rows_bits_are_its_own():
    """A prompt's rows have the same bits whatever lies beside them in their tile: large
    scores in another sequence's rows and NaN among its queries."""
    c = case([40, 50], [20, 30], 200, 4, 1, 128, BF16, 16, seed=11)
    a, la = run(c, max_q=50)
    q = c["q"].clone()
    q[40:] *= 50
    q[41, 2, 3] = float("nan")
    b, lb = run({**c, "q": q}, max_q=50)
    torch.cuda.synchronize()
    assert torch.equal(a[:40], b[:40]) and torch.equal(la[:40], lb[:40])


@pytest.mark.parametrize("D", [128, 256])
def test_same_bits(D):
    """Twice, two at once on two streams, and replayed on other inputs."""
    c, e = (case([40, 1, 90], [300, 5, 90], 460, 4, 2, D, BF16, 16, seed=s) for s in (15, 16))
    d, f = up(c), up(e)
    a, b = run(c, d, max_q=90), run(e, f, max_q=90)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        with torch.cuda.stream(st[0]):
            a2 = run(c, d, max_q=90)
        with torch.cuda.stream(st[1]):
            b2 = run(e, f, max_q=90)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([*a, *b], [*a2, *b2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = run(c, d, max_q=90)
    old = {n: d[n].clone() for n in ("q", "k", "v", "table", "lens", "prefix_pages", "cu")}
    for src, ref in ((f, b), (old, a), (f, b)):
        for n in old:
            d[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(g, ref))
