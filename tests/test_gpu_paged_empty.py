"""Batches of nothing: no tokens of some sequences are a call that does nothing, no
sequences at all are refused, by name."""
import pytest
import torch

from linear_attention_recurrence_fwd_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("S", [0, 2])
def test_no_tokens(S, ragged):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, pools = z(0, 4, 64), z(0, 2, 64), (z(3, 2, 16, 64), z(3, 2, 16, 64))
    cu = i32(S + 1) if ragged else None
    calls = (lambda: B.paged_append(q, k, k, *pools, i32(S, 2), i32(S), cu),
             lambda: B.prefix_attention(q, *pools, i32(S, 2), i32(S), cu=cu),
             lambda: B.prefix_attention(q, *pools, i32(S, 2), i32(S), i32(1), 9, cu))
    for f in calls:
        if S:
            assert f().shape == (0, 4, 64)
        else:
            with pytest.raises(ValueError, match="table: expected a row for each sequence"):
                f()
    torch.cuda.synchronize()
