"""The query/key norm with rotation (gdn_norm_rope_fwd / _bwd, through the
binding) against a 64-bit reference; gradients by torch's autograd through it.

Bounds: an output is rounded once (half a step of its type relative to the
value) after fp32 arithmetic of a few operations on u1 c, u2 s (each at most
|u1| + |u2| large) and a sum of D squares: (D + 16) 2^-24 times those
magnitudes.  dw sums BT H terms in fp32 parts: (BT H + D) 2^-24 times the sum of
their magnitudes."""
import pytest
import torch

import decay_reference as R
from helpers import say
from linear_attention_recurrence_fwd_amd import binding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.lib()


def make(B, T, Hq, Hk, D, Rr, dtype, seed, packed=False, P=64):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s, dt=dtype):
        return torch.randn(s, generator=g).to(dt)
    t = dict(wq=1 + 0.1 * rnd(D, dt=F32), wk=1 + 0.1 * rnd(D, dt=F32), dyq=rnd(B, T, Hq, D), dyk=rnd(B, T, Hk, D))
    if packed:
        x = rnd(B, T, (Hq + 2 * Hk) * D)
        t["q"], t["k"] = x[..., : Hq * D].view(B, T, Hq, D), x[..., Hq * D: (Hq + Hk) * D].view(B, T, Hk, D)
    else:
        t["q"], t["k"] = rnd(B, T, Hq, D), rnd(B, T, Hk, D)
    t["rope"] = binding.rope_table(P, Rr, device="cpu") if Rr else None
    t["pos"] = torch.randint(0, P, (B, T), generator=g).to(torch.int32)
    return t


def up(t, packed):
    c = {n: None if x is None else x.cuda() for n, x in t.items()}
    if packed:  # .cuda() made them dense: cut them out of one tensor again
        B, T, Hq, D = c["q"].shape
        Hk = c["k"].shape[2]
        x = torch.full((B, T, (Hq + 2 * Hk) * D), float("nan"), dtype=c["q"].dtype, device="cuda")
        x[..., : Hq * D] = c["q"].reshape(B, T, -1)
        x[..., Hq * D: (Hq + Hk) * D] = c["k"].reshape(B, T, -1)
        c["q"], c["k"] = x[..., : Hq * D].view(B, T, Hq, D), x[..., Hq * D: (Hq + Hk) * D].view(B, T, Hk, D)
    return c


SIZES = [  # B, T, Hq, Hk, D, R
    (1, 1, 1, 1, 8, 0), (2, 3, 4, 2, 16, 16), (1, 65, 3, 1, 64, 32), (2, 17, 16, 2, 256, 64), (1, 9, 5, 5, 80, 80),
    (2, 33, 8, 8, 128, 128), (1, 130, 6, 3, 192, 64), (1, 5, 2, 2, 512, 512), (3, 7, 1, 1, 104, 48), (1, 40, 33, 1, 32, 0),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_parity(size, dtype, interleaved, packed):
    say("[norm] size=%s dtype=%s interleaved=%d packed=%d" % (size, dtype, interleaved, packed))
    B, T, Hq, Hk, D, Rr = size
    t = make(*size, dtype, 50 + sum(size), packed)
    c = up(t, packed)
    pos = c["pos"] if sum(size) % 2 else None
    tpos = t["pos"] if sum(size) % 2 else None
    if pos is None and T > 64:
        t["rope"] = None if t["rope"] is None else binding.rope_table(T, Rr, device="cpu")
        c["rope"] = None if t["rope"] is None else t["rope"].cuda()
    kw = dict(eps=1e-6, w_offset=0.25, interleaved=interleaved)
    oq, ok = binding.norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["rope"], pos, **kw)
    g = binding.norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["rope"], pos, c["dyq"], c["dyk"], **kw)
    torch.cuda.synchronize()
    z = {n: t[n].double().contiguous().requires_grad_(True) for n in ("q", "k", "wq", "wk")}
    rope = None if t["rope"] is None else t["rope"].double()
    rq, rk = R.norm_rope(z["q"], z["k"], z["wq"], z["wk"], rope, tpos, **kw)
    dyq, dyk = t["dyq"].double(), t["dyk"].double()
    rg = torch.autograd.grad((rq * dyq).sum() + (rk * dyk).sum(), [z[n] for n in ("q", "k", "wq", "wk")])
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    f32 = (D + 16) * 2.0 ** -24
    errs = {}
    for n, got, ref, x in (("oq", oq, rq, "q"), ("ok", ok, rk, "k")):
        xr = z[x].detach()
        r = 1 / torch.sqrt((xr * xr).mean(-1, keepdim=True) + 1e-6)
        mag = 2 * (xr.abs() * r).amax(-1, keepdim=True) * 1.8
        d = (got.double().cpu() - ref.detach()).abs()
        errs[n] = (d / (half * ref.detach().abs() + f32 * mag + 1e-37)).max().item()
    for n, w, x, dy, ref in (("dq", "wq", "q", dyq, rg[0]), ("dk", "wk", "k", dyk, rg[1])):
        xr = z[x].detach()
        r = 1 / torch.sqrt((xr * xr).mean(-1, keepdim=True) + 1e-6)
        e = 2 * dy.abs().amax(-1, keepdim=True) * 1.8
        mag = r * (e + (xr.abs() * r) * e * (xr.abs() * r).mean(-1, keepdim=True))
        d = (g[n].double().cpu() - ref).abs()
        errs[n] = (d / (half * ref.abs() + f32 * mag + 1e-37)).max().item()
        # the weights' gradients
        rw = rg[2] if n == "dq" else rg[3]
        H = xr.shape[2]
        magw = (xr.abs() * r * 2 * dy.abs().amax(-1, keepdim=True)).sum((0, 1, 2))
        d = (g["dw" + n[1]].double().cpu() - rw).abs()
        errs["dw" + n[1]] = (d / ((B * T * H + D + 16) * 2.0 ** -24 * magw + 1e-37)).max().item()
    say("[norm] share of the bounds: " + " ".join("%s=%.2f" % kv for kv in errs.items()))
    assert all(e <= 1.0 for e in errs.values()), errs
    assert oq.is_contiguous() and ok.is_contiguous()


def test_bad_positions_are_nan():
    """A position outside the table turns the first R channels of its token to
    NaN, nothing else."""
    t = make(1, 6, 2, 2, 64, 32, F32, 9, P=16)
    c = up(t, False)
    good = c["pos"].clone()
    c["pos"][0, 2], c["pos"][0, 4] = 16, -1
    oq, ok = binding.norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["pos"])
    rq, rk = binding.norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["rope"], good)
    for o, r in ((oq, rq), (ok, rk)):
        for i in (2, 4):
            assert torch.isnan(o[0, i, :, :32]).all() and torch.equal(o[0, i, :, 32:], r[0, i, :, 32:])
        keep = [0, 1, 3, 5]
        assert torch.equal(o[0, keep], r[0, keep])


def test_nan_and_zero_rows_stay_in_their_rows():
    t = make(1, 4, 3, 2, 128, 128, BF, 4)
    c = up(t, False)
    ref = binding.norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["pos"])[0]
    c["q"][0, 1, 1] = float("nan")
    c["q"][0, 2, 0] = 0
    o = binding.norm_rope(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["pos"])[0]
    assert torch.isnan(o[0, 1, 1]).all() and (o[0, 2, 0] == 0).all()
    keep = torch.ones((4, 3), dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = False
    assert torch.equal(o[0][keep.cuda()], ref[0][keep.cuda()])


def test_repeats_are_bitwise():
    t = make(2, 300, 6, 2, 128, 64, BF, 8)
    c = up(t, False)
    a = binding.norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["pos"], c["dyq"], c["dyk"])
    b = binding.norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["rope"], c["pos"], c["dyq"], c["dyk"])
    for n in a:
        assert torch.equal(a[n].view(torch.uint8) if a[n].dtype == BF else a[n],
                           b[n].view(torch.uint8) if b[n].dtype == BF else b[n]), n
