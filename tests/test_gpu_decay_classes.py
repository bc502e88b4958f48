"""The decay operator at every class of head sizes and in segments of several
chunks: the segments' sums, their prefix in the walks (up to eight segments) and the
chain over them (more, or a state updated in place), both directions, against the
64-bit recurrences (decay_recurrence, itself held to the step-by-step reference's
autograd here)."""
import pytest
import torch

import decay_reference as R
from decay_recurrence import check_call, recurrence
from helpers import say
from linear_attention_recurrence_fwd_amd import binding

BF, F32 = torch.bfloat16, torch.float32


def make(B, T, Hk, Hv, Dk, Dv, dtype, seed, mask, device="cuda", slow=10.0):
    g = torch.Generator(device=device).manual_seed(seed)

    def rnd(*s, dt=dtype):
        return torch.randn(s, generator=g, device=device).to(dt)
    t = dict(q=rnd(B, T, Hk, Dk), k=rnd(B, T, Hk, Dk), v=rnd(B, T, Hv, Dv), dO=rnd(B, T, Hv, Dv),
             lg=-torch.exp2(-slow * torch.rand((Hv,), generator=g, device=device)),
             state0=rnd(B, Hv, Dk, Dv, dt=F32), dS=rnd(B, Hv, Dk, Dv, dt=F32), mask=None)
    if mask != "none":
        at = torch.arange(T, device=device)[None]
        n = torch.randint(T // 4, T + 1, (B, 1), generator=g, device=device)
        if B > 1:
            n[0] = 0  # one sequence without a valid step
        m = at < n if mask == "behind" else at >= T - n if mask == "before" else \
            torch.rand((B, T), generator=g, device=device) < 0.6
        t["mask"] = m.to(torch.uint8)
        for x in ("k", "v"):  # what stands at masked steps is not read
            t[x][~m] = float("nan")
    return t


@pytest.mark.parametrize("mask", ["none", "some", "behind"])
def test_recurrence_is_the_reference(mask):
    """fp64 against fp64: sums of at most a few hundred terms, 1e-12 of the largest value."""
    t = make(2, 9, 2, 4, 16, 8, torch.float64, 3, mask, "cpu", slow=2.0)
    t = {n: None if x is None else x if n == "mask" else x.double() for n, x in t.items()}
    got = recurrence(t["q"], t["k"], t["v"], t["lg"], t["state0"], t["mask"], t["dO"], t["dS"], 0.3)
    k, v = R.clean(t["k"], t["v"], t["mask"])
    o, st = R.decay(t["q"], k, v, t["lg"], t["state0"], t["mask"], 0.3)
    ref = dict(R.decay_grads(t["q"], k, v, t["lg"], t["state0"], t["mask"], t["dO"], t["dS"], 0.3), o=o, state=st)
    for n in ref:
        assert (got[n] - ref[n]).abs().max() <= 1e-12 * ref[n].abs().max(), n


def run(t, tag, segments, in_place=False, bwd=True):
    B, T, Hk, Dk = t["q"].shape
    Hv, Dv = t["v"].shape[2:]
    say("[classes] " + tag)
    d = binding.make_dims(B, T, Hk, Hv, Dk, Dv, t["q"].dtype)
    if segments:  # (one pass asks for no workspace)
        assert binding._query("gdn_decay_fwd_workspace_bytes", d) > 0
    got = {}
    s = t["state0"].clone()
    got["o"], got["state"] = binding.decay_fwd(t["q"], t["k"], t["v"], t["lg"], s, t["mask"], state_out=s if in_place else None)
    torch.cuda.synchronize()
    say("[classes] forward done")
    if bwd:
        got.update(binding.decay_bwd(t["q"], t["k"], t["v"], t["lg"], t["state0"], t["mask"], t["dO"], t["dS"]))
        torch.cuda.synchronize()
        say("[classes] backward done")
    errs = check_call(t, got)
    say("[classes] " + " ".join("%s=%.1e" % kv for kv in errs.items()))


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()


name = lambda s: "x".join(map(str, s))  # noqa: E731

# every class of Dk with Dv in 129 .. 192, and those of Dv with Dk in 193 .. 256, with one,
# two and three value heads to a key head
CLASSES = [
    (1, 150, 1, 2, 40, 136), (2, 97, 1, 3, 128, 160), (1, 130, 2, 4, 192, 192), (1, 100, 1, 1, 256, 184), (2, 70, 1, 1, 96, 176),
    (1, 140, 1, 2, 136, 144), (1, 90, 1, 2, 200, 24), (1, 150, 1, 3, 224, 112), (2, 65, 1, 2, 248, 256), (1, 190, 2, 2, 192, 256),
    (1, 129, 1, 2, 64, 240), (1, 66, 1, 2, 128, 208), (1, 200, 1, 2, 160, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("mask", ["none", "some"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", CLASSES, ids=name)
def test_classes_of_head_sizes(size, dtype, mask):
    gpu()
    run(make(*size, dtype, 7 + sum(size), mask), "%s %s %s" % (size, dtype, mask), False)


# eight segments or fewer, of three to eight chunks; and sixteen of four
PREFIX = [
    (1, 2040, 4, 32, 192, 128), (2, 2040, 16, 16, 128, 128), (1, 2040, 16, 32, 128, 192), (2, 1025, 8, 16, 256, 256),
    (1, 1530, 11, 33, 72, 200), (3, 2040, 4, 16, 200, 136), (1, 2040, 16, 32, 64, 256), (4, 2047, 8, 16, 192, 128),
    (1, 1990, 16, 32, 256, 40),
]
CHAIN = [(1, 4090, 4, 16, 192, 128), (2, 4090, 4, 8, 128, 128), (1, 3970, 8, 16, 128, 176), (1, 4090, 15, 15, 224, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mask", ["none", "some", "behind", "before"])
@pytest.mark.parametrize("size", PREFIX, ids=name)
def test_few_segments_of_several_chunks(size, mask, dtype):
    gpu()
    run(make(*size, dtype, 7 + sum(size), mask), "%s %s %s" % (size, dtype, mask), True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", PREFIX, ids=name)
def test_few_segments_in_place(size, dtype):
    gpu()
    run(make(*size, dtype, 9 + sum(size), "some"), "in place %s %s" % (size, dtype), True, in_place=True, bwd=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mask", ["none", "some"])
@pytest.mark.parametrize("size", CHAIN, ids=name)
def test_many_segments_of_several_chunks(size, mask, dtype):
    gpu()
    run(make(*size, dtype, 7 + sum(size), mask), "%s %s %s" % (size, dtype, mask), True)
