"""The query/key norm with rotation (through the binding) over many tokens, against
64 bits at stretches of them (on the GPU), with the bounds of test_gpu_norm_rope:
half a step of the type relative to the value, and (D + 16) 2^-24 times the
magnitudes that the fp32 arithmetic adds up."""
import pytest
import torch

import decay_reference as R
from helpers import say
from linear_attention_recurrence_fwd_amd import binding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
KW = dict(eps=1e-6, w_offset=0.25)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()


def make(B, T, Hq, Hk, D, Rr, dtype, seed, packed, P=64):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s, dt=dtype):
        return torch.randn(s, generator=g, device="cuda", dtype=dt)
    c = dict(wq=1 + 0.1 * rnd(D, dt=F32), wk=1 + 0.1 * rnd(D, dt=F32), dyq=rnd(B, T, Hq, D), dyk=rnd(B, T, Hk, D))
    if packed:
        x = rnd(B, T, (Hq + 2 * Hk) * D)
        c["q"], c["k"] = x[..., : Hq * D].view(B, T, Hq, D), x[..., Hq * D: (Hq + Hk) * D].view(B, T, Hk, D)
    else:
        c["q"], c["k"] = rnd(B, T, Hq, D), rnd(B, T, Hk, D)
    c["rope"] = binding.rope_table(P, Rr) if Rr else None
    c["pos"] = torch.randint(0, P, (B, T), generator=g, device="cuda", dtype=torch.int32)
    return c


def shares(c, outs, grads, b, s, interleaved):
    """Shares of the bounds that outputs and gradients of tokens s of sequence b take."""
    cut = lambda x: x[b:b + 1, s]  # noqa: E731
    w = [c[n].double() for n in ("wq", "wk")]
    z = [cut(c[n]).double().requires_grad_(True) for n in ("q", "k")]
    rope = None if c["rope"] is None else c["rope"].double()
    ref = R.norm_rope(*z, *w, rope, cut(c["pos"]), interleaved=interleaved, **KW)
    dy = [cut(c[n]).double() for n in ("dyq", "dyk")]
    rg = torch.autograd.grad(sum((r * d).sum() for r, d in zip(ref, dy)), z)
    D = z[0].shape[-1]
    half, f32 = 2.0 ** -8 if c["q"].dtype == BF else 2.0 ** -24, (D + 16) * 2.0 ** -24
    e = {}
    for i, n in enumerate("qk"):
        x = z[i].detach()
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        mag = 2 * (x.abs() * r).amax(-1, keepdim=True) * 1.8
        e["o" + n] = ((cut(outs[i]).double() - ref[i].detach()).abs() / (half * ref[i].detach().abs() + f32 * mag)).max().item()
        a = 2 * dy[i].abs().amax(-1, keepdim=True) * 1.8
        mag = r * (a + (x.abs() * r) * a * (x.abs() * r).mean(-1, keepdim=True))
        e["d" + n] = ((cut(grads["d" + n]).double() - rg[i]).abs() / (half * rg[i].abs() + f32 * mag)).max().item()
    return e


def weights(c, grads, interleaved):
    """Shares of their bound that the weights' gradients take: sums over all rows,
    here in 64 bits over runs of tokens; each off by at most (B T H + D + 16) 2^-24
    times its terms' magnitudes.  Normwise the roundings are independent and the terms
    of either sign: (D + 16) 2^-24 for the terms themselves and the root of their
    number times 2^-24 for the sums, eight times that for what a partial sum may be
    larger than the whole."""
    e = {}
    B, T, _, D = c["q"].shape
    rope = None if c["rope"] is None else c["rope"].double()
    wq, wk = (c[n].double().requires_grad_(True) for n in ("wq", "wk"))
    sums, mags = [0.0, 0.0], [0.0, 0.0]
    run = max(1, (1 << 22) // c["q"].shape[2] // D)
    for b in range(B):
        for t in range(0, T, run):
            cut = lambda x: x[b:b + 1, t:t + run].double()  # noqa: E731
            ref = R.norm_rope(cut(c["q"]), cut(c["k"]), wq, wk, rope, c["pos"][b:b + 1, t:t + run], interleaved=interleaved, **KW)
            g = torch.autograd.grad((ref[0] * cut(c["dyq"])).sum() + (ref[1] * cut(c["dyk"])).sum(), [wq, wk])
            for i, n in enumerate("qk"):
                x = cut(c[n])
                r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
                sums[i] = sums[i] + g[i]
                mags[i] = mags[i] + (x.abs() * r * 2 * cut(c["dy" + n]).abs().amax(-1, keepdim=True)).sum((0, 1, 2))
    for i, n in enumerate("qk"):
        terms = B * T * c[n].shape[2] + D + 16
        d = grads["dw" + n].double() - sums[i]
        e["dw" + n] = (d.abs() / (terms * 2.0 ** -24 * mags[i])).max().item()
        e["dw" + n + " norm"] = (d.norm() / sums[i].norm() / (8 * (D + 16 + terms ** 0.5) * 2.0 ** -24)).item()
    return e


@pytest.mark.parametrize("size", [(1, (1 << 24) + 9, 2, 1, 16, 16), (3, (1 << 24) + 5, 1, 1, 8, 0), (1, (1 << 26) + 9, 1, 1, 8, 0)],
                         ids=lambda s: "x".join(map(str, s)))
def test_more_tokens_than_one_direction_of_a_grid(size):
    """From 2^24 tokens the forward's workgroups go on in the grid's second direction;
    from 2^26 their threads would be more than one direction holds."""
    say("[norm long] size=%s" % (size,))
    c = make(*size, BF, 3, False)
    outs = binding.norm_rope(*[c[n] for n in ("q", "k", "wq", "wk", "rope", "pos")], **KW)
    torch.cuda.synchronize()
    say("[norm long] forward done")
    g = binding.norm_rope_bwd(*[c[n] for n in ("q", "k", "wq", "wk", "rope", "pos", "dyq", "dyk")], **KW)
    torch.cuda.synchronize()
    say("[norm long] backward done")
    B, T = size[:2]
    for b in {0, B - 1}:
        for t in (0, (1 << 23) - 500, (1 << 24) - 600, T // 2, T - 1000):
            e = shares(c, outs, g, b, slice(t, t + 1000), False)
            assert all(x <= 1.0 for x in e.values()), (b, t, e)


# B, T, Hq, Hk, D, R.  A wave takes 64 / lanes heads of a token at a time (lanes of eight
# channels, a power of two) and a run of such groups: with so many tokens runs of two
# and more, of which one has query and key heads, up to all heads of a token; and the
# backward's waves take several of these.
PROMPTS = [
    (1, 3001, 20, 12, 128, 128), (2, 1500, 17, 7, 128, 64), (1, 2500, 7, 4, 256, 64), (3, 3333, 24, 9, 64, 32),
    (1, 9001, 5, 2, 192, 192), (1, 2100, 6, 5, 512, 512), (1, 9000, 70, 65, 8, 0), (2, 5000, 40, 3, 40, 32),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", PROMPTS, ids=lambda s: "x".join(map(str, s)))
def test_prompts(size, dtype, interleaved, packed):
    say("[norm prompt] size=%s dtype=%s interleaved=%d packed=%d" % (size, dtype, interleaved, packed))
    c = make(*size, dtype, sum(size), packed)
    kw = dict(KW, interleaved=interleaved)
    outs = binding.norm_rope(*[c[n] for n in ("q", "k", "wq", "wk", "rope", "pos")], **kw)
    g = binding.norm_rope_bwd(*[c[n] for n in ("q", "k", "wq", "wk", "rope", "pos", "dyq", "dyk")], **kw)
    torch.cuda.synchronize()
    for b in range(size[0]):
        e = shares(c, outs, g, b, slice(0, size[1]), interleaved)
        assert all(x <= 1.0 for x in e.values()), (b, e)
    e = weights(c, g, interleaved)
    say("[norm prompt] shares of the weights' bounds: " + " ".join("%s=%.3f" % kv for kv in e.items()))
    assert all(x <= 1.0 for x in e.values()), e


@pytest.mark.parametrize("Rr", [0, 32])
def test_no_tokens(Rr):
    """No rows: empty outputs, zero gradients of the weights."""
    c = make(2, 0, 3, 2, 64, Rr, BF, 4, False)
    for pos in (None, c["pos"]):
        oq, ok = binding.norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["rope"], pos, **KW)
        g = binding.norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["rope"], pos, c["dyq"], c["dyk"], **KW)
        torch.cuda.synchronize()
        assert oq.shape == g["dq"].shape == (2, 0, 3, 64) and ok.shape == g["dk"].shape == (2, 0, 2, 64)
        assert (g["dwq"] == 0).all() and (g["dwk"] == 0).all()
