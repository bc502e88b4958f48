"""Attention over a shared prefix where scores are enormous, infinite or NaN: a call of
any values ends, and what can be said of the result holds."""
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


def pool(keys, Hk, D, dtype, seed, n_seq):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    k, v = rnd(keys // 16 + n_seq, Hk, 16, D), rnd(keys // 16 + n_seq, Hk, 16, D)
    prefix = torch.arange(keys // 16, dtype=torch.int32, device="cuda")
    table = torch.arange(keys // 16, keys // 16 + n_seq, dtype=torch.int32, device="cuda").view(n_seq, 1)
    lens = torch.full((n_seq,), 3, dtype=torch.int32, device="cuda")
    return k, v, prefix, table, lens


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e9, 1e15, 1e25, 1e36])
def test_one_key_far_above_the_others(dtype, rows, size):
    """Scores of +-size: all but the keys of the largest score have weight 0, however the
    scores' last bits fall; here one key of the prefix has twice the others' size."""
    n_seq, Hk, D, keys = rows, 1, 64, 640
    k, v, prefix, table, lens = pool(keys, Hk, D, dtype, 1, n_seq)
    k.zero_()
    k[:, :, :, 0] = 1.0
    k[7, 0, 5, 0] = 2.0
    q = torch.zeros((n_seq, 4, D), dtype=dtype, device="cuda")
    q[:, :, 0] = size
    o = B.prefix_attention(q, k, v, table, lens, prefix, keys, scale=1.0)
    torch.cuda.synchronize()
    assert torch.equal(o, v[7, 0, 5].expand_as(o))
    # and with the sign turned every other key ties: their mean
    o = B.prefix_attention(q, k, v, table, lens, prefix, keys, scale=-1.0)
    torch.cuda.synchronize()
    others = torch.cat([x for i, x in enumerate(v[: keys // 16, 0].double().reshape(-1, D).unbind()) if i != 7 * 16 + 5]).view(-1, D)
    own = v[keys // 16:, 0, :3].double()
    mean = (others.sum(0) + own.sum(1)) / (keys - 1 + 3)
    assert (o.double() - mean[:, None]).abs().max() < (2e-2 if dtype == torch.bfloat16 else 1e-5)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_that_are_no_numbers(dtype, rows):
    """Infinite and NaN keys and queries: those rows are NaN, the others as without them."""
    n_seq, Hk, D, keys = rows, 1, 64, 320
    k, v, prefix, table, lens = pool(keys, Hk, D, dtype, 2, n_seq)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((n_seq, 4, D), generator=g, device="cuda").to(dtype)
    ref = B.prefix_attention(q, k, v, table, lens, prefix, keys)
    x = q.clone()
    x[0, 0, 3], x[0, 1, 4], x[-1, 3, 5] = math.nan, math.inf, -math.inf
    o = B.prefix_attention(x, k, v, table, lens, prefix, keys)
    torch.cuda.synchronize()
    bad = torch.zeros((n_seq, 4), dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[0, 1] = bad[-1, 3] = True
    assert torch.isnan(o[bad].float()).all() and torch.equal(o[~bad], ref[~bad])
    for value in (math.nan, math.inf, -math.inf):
        y = k.clone()
        y[3, 0, 2, 1] = value
        o = B.prefix_attention(q, y, v, table, lens, prefix, keys)
        torch.cuda.synchronize()
        if math.isnan(value):
            assert torch.isnan(o.float()).all()
        else:
            up = (q[..., 1].float() * value) > 0  # a score of +inf: no weights; of -inf: a key without weight
            assert torch.isnan(o[up].float()).all() and torch.isfinite(o[~up].float()).all()
