"""The tests' 64-bit forms of the rotation with several axes and of the attention: the
gradient formulas against differences, the attention against another way to it."""
import math

import pytest
import torch

import paged_reference as R


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_gradients_against_differences(norm, interleaved):
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    tokens, H, D, rot = 3, 2, 24, 16
    rope = torch.cat([torch.cos(rnd(9, rot // 2)), torch.sin(rnd(9, rot // 2))], 1)
    axis, pos = torch.randint(0, 3, (rot // 2,), generator=g), torch.randint(0, 9, (3, tokens), generator=g)
    z = R.turns(rope, axis, pos)
    x, w, dy = rnd(tokens, H, D), (1 + 0.1 * rnd(D)) if norm else None, rnd(tokens, H, D)
    dx, dw, _, _ = R.norm_turn_vjp(x, w, z, dy, rot, interleaved, 1e-3, 0.25)

    def loss(x, w):
        return (R.norm_turn(x, w, z, rot, interleaved, 1e-3, 0.25)[0] * dy).sum()

    h = 1e-6
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        diff = (loss(x + e.view_as(x), w) - loss(x - e.view_as(x), w)) / (2 * h)
        assert abs(diff - dx.view(-1)[i]) < 1e-7 * (1 + abs(diff))
    if norm:
        for i in range(D):
            e = torch.zeros_like(w)
            e[i] = h
            diff = (loss(x, w + e) - loss(x, w - e)) / (2 * h)
            assert abs(diff - dw[i]) < 1e-7 * (1 + abs(diff))


def test_rotation_is_by_the_pair_s_own_axis():
    rope = torch.cat([torch.tensor([[1.0, 1.0], [0.0, 0.0]]), torch.tensor([[0.0, 0.0], [1.0, 1.0]])], 1)  # 0 and 90 degrees
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 9.0]]], dtype=torch.float64)
    for pos, want in (([[0], [0]], [1, 2, 3, 4, 9]), ([[1], [0]], [-3, 2, 1, 4, 9]), ([[0], [1]], [1, -4, 3, 2, 9])):
        z = R.turns(rope, torch.tensor([0, 1]), torch.tensor(pos))
        assert torch.equal(R.rotate(x, z, 4, False)[0, 0], torch.tensor(want, dtype=torch.float64))


@pytest.mark.parametrize("prefix", [0, 5])
def test_attention_by_padded_masks(prefix):
    """Against all keys side by side with a mask and torch's softmax."""
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    Hk, G, D, page, new, lens = 2, 2, 8, 4, [2, 3], [6, 3]
    k, v = rnd(9, Hk, page, D), rnd(9, Hk, page, D)
    table, pages = torch.tensor([[3, 1], [7, 0]]), torch.tensor([5, 2])
    q = rnd(5, Hk * G, D).float()
    o, lse, _, _ = R.attention(q, k, v, table, torch.tensor(lens), pages, prefix, torch.tensor([0, 2, 5]), 0.7)
    for s in range(2):
        ids = torch.cat([pages, table[s]])
        kk, vv = (x[ids].permute(1, 0, 2, 3).reshape(Hk, -1, D) for x in (k, v))
        place = torch.arange(4 * page)
        for t in range(new[s]):
            row = [0, 2][s] + t
            own = place - 2 * page
            seen = (place < prefix) | ((own >= 0) & (own <= lens[s] - new[s] + t))
            a = torch.einsum("hgd,hkd->hgk", q[row].double().view(Hk, G, D), kk) * 0.7
            a = a.masked_fill(~seen, -math.inf)
            assert torch.allclose(o[row].view(Hk, G, D), torch.softmax(a, -1) @ vv, atol=1e-12)
            assert torch.allclose(lse[row].view(Hk, G), torch.logsumexp(a, -1), atol=1e-12)
