"""Many steps in turn with slow decays (the per-step form, and single tokens one call
after the other, in place), against the 64-bit recurrence.

Bound, normwise.  A step rounds the state once or twice, 2^-24 of it each, in either
direction; a state remembers n = min(T, 1/|lg|) steps, so their sum is sqrt(n) 2^-24
of it, taken five times as in decay_recurrence for what cancels; 1e-6 for the
exponential and the products of a few steps.  (A decay that is itself off by 2^-25
gives n 2^-25, twenty times that.)"""
import pytest
import torch

from decay_recurrence import recurrence
from helpers import say
from linear_attention_recurrence_fwd_amd import binding

pytestmark = pytest.mark.gpu
LG = [-2.0 ** -6, -2.0 ** -8 * 1.1, -2.0 ** -10 * 1.3, -2.0 ** -12 * 1.2, -2.0 ** -13 * 1.7, -1e-5, 0.0, 2.0 ** -14]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()


def inputs(T, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hv = len(LG)
    r = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    return r(1, T, 1, 24), r(1, T, 1, 24), r(1, T, Hv, 40), torch.tensor(LG, device="cuda")


def bound(lg, T):
    return 5 * min(T, 1 / abs(lg) if lg else T) ** 0.5 * 2.0 ** -24 + 1e-6


@pytest.mark.parametrize("seed", [1, 2])
def test_states_of_many_steps(seed):
    T = 20000
    q, k, v, lg = inputs(T, seed)
    o, st = binding.decay_fwd(q, k, v, lg, algo=binding.ALGO_SCAN)
    torch.cuda.synchronize()
    say("[decode] %d steps done" % T)
    ref = recurrence(q.double(), k.double(), v.double(), lg.double(), None, None)
    last = slice(T - 1000, T)
    for h, x in enumerate(LG):
        for n, a, b in (("state", st[:, h], ref["state"][:, h]), ("o", o[:, last, h], ref["o"][:, last, h])):
            e = ((a.double() - b).norm() / b.norm()).item()
            say("[decode] lg=%.1e %s %.1e of %.1e" % (x, n, e, bound(x, T)))
            assert e <= bound(x, T), (x, n)


def test_single_tokens_in_place():
    T = 3000
    q, k, v, lg = inputs(T, 5)
    s = torch.zeros((1, len(LG), 24, 40), device="cuda")
    for t in range(T):
        binding.decay_fwd(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], lg, s, state_out=s)
    ref = recurrence(q.double(), k.double(), v.double(), lg.double(), None, None)["state"]
    for h, x in enumerate(LG):
        e = ((s[:, h].double() - ref[:, h]).norm() / ref[:, h].norm()).item()
        say("[decode] tokens lg=%.1e %.1e of %.1e" % (x, e, bound(x, T)))
        assert e <= bound(x, T), x
