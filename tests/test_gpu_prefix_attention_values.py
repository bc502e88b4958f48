"""Attention over a shared prefix and own pages where values are enormous or tiny: a result
that the type holds is not lost on the way, whatever the order in which scores grow."""
import math

import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def attend(score, value, own, rows, dtype, D=64, scale=math.log(2)):
    """rows single tokens over a prefix of the given scores (base 2: the scale times log2 e
    is 1 in fp32) and values, and `own` own keys of the same; (o, lse)."""
    def pool(n):
        pages = -(-n // 16)
        k = torch.zeros((pages, 1, 16, D), dtype=dtype, device="cuda")
        v = torch.zeros_like(k)
        k.view(-1, D)[:n, 0] = score[:n].to(dtype).cuda()
        v.view(-1, D)[:n] = value[:n].to(dtype).cuda()[:, None]
        return k, v

    n = score.numel()
    (k, v), (ko, vo) = pool(n), pool(own)
    prefix = torch.arange(k.shape[0], dtype=torch.int32, device="cuda")
    table = torch.arange(k.shape[0], k.shape[0] + ko.shape[0], dtype=torch.int32, device="cuda").expand(rows, -1).contiguous()
    lens = torch.full((rows,), own, dtype=torch.int32, device="cuda")
    q = torch.zeros((rows, 4, D), dtype=dtype, device="cuda")
    q[:, :, 0] = 1
    o, lse = B.prefix_attention(q, torch.cat([k, ko]), torch.cat([v, vo]), table, lens, prefix, n, scale=scale, lse=True)
    torch.cuda.synchronize()
    return o.double().cpu(), lse.double().cpu()


def reference(score, value, own):
    s, v = torch.cat([score, score[:own]]).double(), torch.cat([value, value[:own]]).double()
    p = torch.softmax(s * math.log(2), 0)
    return float((p * v).sum()), float(torch.logsumexp(s * math.log(2), 0))


def tolerance(dtype, n):
    """Relative, of values of one sign: the exponent's rounding (under 64 in size: 2^-19 of it,
    2^-19.5 of the weight), sums of n terms in parts, a bf16 weight's and the result's rounding."""
    return 2.0 ** -19 + (n / 8 + 64) * 2.0 ** -24 + (2 * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0)


@DTYPES
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("size", [1e34, 1e37, 3e38])
@pytest.mark.parametrize("step", [0, 6, 15])
def test_enormous_values(dtype, rows, size, step):
    """Values near the type's largest behind scores that are equal, or grow by a little less
    than what moves the softmax's reference: many weights above the first key's."""
    n = 1600
    score = torch.full((n,), float(step))
    score[0] = 0
    value = torch.full((n,), size).to(dtype).float()
    for own in (1, 17):
        o, lse = attend(score, value, own, rows, dtype)
        ref, ref_lse = reference(score, value, own)
        t = tolerance(dtype, n)
        assert torch.isfinite(o).all()
        assert ((o - ref).abs() <= t * ref).all(), (o.max(), ref)
        assert ((lse - ref_lse).abs() <= t + 4 * 2.0 ** -24 * abs(ref_lse)).all()


@DTYPES
@pytest.mark.parametrize("rows", [1, 40])
def test_enormous_values_behind_enormous_scores(dtype, rows):
    """The same beside scores of 2^21 and of 2^28, where a step of a score's last bit is
    more than any bound of the weights."""
    for top in (2.0 ** 21, 2.0 ** 28):
        n = 800
        score = torch.full((n,), top / 2)
        score[300:] = top
        value = torch.full((n,), 1e38).to(dtype).float()
        o, _ = attend(score, value, 3, rows, dtype)
        ref, _ = reference(score, value, 3)
        assert torch.isfinite(o).all() and ((o - ref).abs() <= tolerance(dtype, n) * ref).all()


@DTYPES
@pytest.mark.parametrize("rows", [1, 40])
def test_tiny_values(dtype, rows):
    """Values of 1e-27: the products stay above fp32's smallest normal number."""
    n = 1600
    score = torch.linspace(-3, 3, n).to(torch.bfloat16).float()
    value = torch.full((n,), 1e-27).to(dtype).float()
    o, _ = attend(score, value, 5, rows, dtype)
    ref, _ = reference(score, value, 5)
    assert ((o - ref).abs() <= tolerance(dtype, n) * ref).all()


@DTYPES
@pytest.mark.parametrize("rows", [1, 40])
def test_values_of_both_signs(dtype, rows):
    """Enormous values that cancel: finite, and within the weights' roundings of their size."""
    n = 1600
    score = torch.where(torch.arange(n) == 0, 0.0, 15.0)
    value = (torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0) * 1e38).to(dtype).float()
    o, _ = attend(score, value, 4, rows, dtype)
    ref, _ = reference(score, value, 4)
    assert torch.isfinite(o).all() and ((o - ref).abs() <= tolerance(dtype, n) * 1e38).all()
