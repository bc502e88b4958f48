"""Growth (lg > 0) over many segments, up to where g^n still is a number: against the
64-bit reference, with the bounds of decay_reference (relative to what is added up,
which grows alike)."""
import pytest
import torch

import decay_reference as R
from helpers import say
from linear_attention_recurrence_fwd_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("algo", [binding.ALGO_CHUNK, binding.ALGO_CHUNK_TPAR])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_growth_up_to_the_largest_power(dtype, algo):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("[decay growth] %s algo=%d" % (dtype, algo))
    B, T, Hk, Hv, Dk, Dv = 1, 1500, 1, 2, 64, 40
    g = torch.Generator().manual_seed(2)
    r = lambda *s, dt=dtype: torch.randn(s, generator=g).to(dt)  # noqa: E731
    q, k, v = r(B, T, Hk, Dk), r(B, T, Hk, Dk), r(B, T, Hv, Dv)
    lg = torch.tensor([70.0 / T, 20.0 / T])  # g^T = e^70 and e^20, with states of a few hundred times that
    o, st = binding.decay_fwd(q.cuda(), k.cuda(), v.cuda(), lg.cuda(), algo=algo)
    torch.cuda.synchronize()
    x = [t.double() for t in (q, k, v)]
    ro, rst = R.decay(*x, lg.double())
    mo, mst = R.decay(*[t.abs() for t in x], lg.double())
    # the exponents reach 101 (in powers of two), where a step of 2^-24 of them is 101 ln 2 steps of the power
    terms = Dk + Dv + 128 + T + 71
    rounded = dtype == torch.bfloat16
    R.check("o", o, ro, mo, dtype, terms, rounded)
    R.check("state", st, rst, mst, dtype, terms, False)
