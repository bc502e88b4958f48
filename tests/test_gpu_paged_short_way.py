"""The short way (_calls) is what runs: it answers every call that it is meant for, with
tensors of its own kind, and its answer is the long way's."""
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


class Recorder:
    """_calls, with what each of its functions answered."""

    def __init__(self, calls):
        self.calls, self.answers = calls, []

    def __getattr__(self, name):
        def call(*args):
            self.answers.append((name, getattr(self.calls, name)(*args)))
            return self.answers[-1][1]
        return call


def flat(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [z for y in (x.values() if isinstance(x, dict) else x) if y is not None for z in flat(y)]


def short(monkeypatch, name, f):
    """f's result, which the short way's function of this name has to have given, and which
    has to be the long way's."""
    assert B._calls is not None
    recorder = Recorder(B._calls)
    monkeypatch.setattr(B, "_calls", recorder)
    a = f()
    assert [n for n, _ in recorder.answers] == [name]
    assert recorder.answers[0][1] is not NotImplemented and recorder.answers[0][1] is a
    monkeypatch.setattr(B, "_calls", None)
    b = f()
    monkeypatch.undo()
    torch.cuda.synchronize()
    x, y = flat(a), flat(b)
    assert len(x) == len(y) and all(s.dtype == t.dtype and s.stride() == t.stride() and torch.equal(s, t) for s, t in zip(x, y))
    return a


@DTYPES
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("axes", [None, 1, 2, 4])
@pytest.mark.parametrize("rotated", [False, True])
def test_rotation(monkeypatch, dtype, packed, norm, axes, rotated):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, 5, 6, 64), generator=g, device="cuda").to(dtype)
    q, k = x[:, :, :4], x[:, :, 4:]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    wq, wk = [1 + torch.randn(64, generator=g, device="cuda") / 8 for _ in range(2)] if norm else (None, None)
    rope = B.rope_table(32, 32) if rotated else None
    pos = None if axes is None else torch.randint(0, 30, (axes, 2, 5), generator=g, device="cuda", dtype=torch.int32)
    axis = B.axis_map([16 // axes] * axes) if axes and rotated else None
    kw = dict(axis=axis, pos=pos, eps=1e-5, w_offset=0.5, interleaved=packed)
    y = short(monkeypatch, "norm_rope_axes", lambda: B.norm_rope_axes(q, k, wq, wk, rope, **kw))
    short(monkeypatch, "norm_rope_axes_bwd", lambda: B.norm_rope_axes_bwd(q, k, wq, wk, rope, dyq=y[0], dyk=y[1], **kw))


@DTYPES
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("beside", [False, True])
def test_append(monkeypatch, dtype, ragged, beside):
    """Packed rows, with and without cu, queries, the norm, a rotation, positions, out."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((6, 8, 64), generator=g, device="cuda").to(dtype)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    w = [1 + torch.randn(64, generator=g, device="cuda") / 8 for _ in range(2)]
    table = torch.tensor([[3, 0], [2, 1]], dtype=torch.int32, device="cuda")
    past = torch.tensor([3, 15], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda") if ragged else None
    rope, axis = B.rope_table(40, 32), B.axis_map([8, 8])
    pos = torch.randint(0, 40, (2, 6), generator=g, device="cuda", dtype=torch.int32)
    turned = dict(wq=w[0], wk=w[1], rope=rope, first=2, eps=1e-5, w_offset=0.5, interleaved=beside)
    calls = [dict(turned), dict(turned, axis=axis, pos=pos), dict(wq=w[0], wk=w[1]), dict(rope=rope), dict()]

    def run(queries=True, out=None, **kw):
        if beside:
            both = torch.zeros((4, 2, 2, 16, 64), dtype=dtype, device="cuda")
            kp, vp = both[:, 0], both[:, 1]
        else:
            kp, vp = (torch.zeros((4, 2, 16, 64), dtype=dtype, device="cuda") for _ in range(2))
        pools.append((kp, vp))
        return B.paged_append(q if queries else None, k, v, kp, vp, table, past, cu, out=out, **kw)

    for kw in calls:
        pools = []
        short(monkeypatch, "paged_append", lambda: run(**kw))
        assert all(torch.equal(a, b) and a.any() for a, b in zip(*pools))
    into = torch.empty((6, 4, 64), dtype=dtype, device="cuda")
    pools = []
    assert short(monkeypatch, "paged_append", lambda: run(out=into, **calls[0])) is into
    # without queries there is nothing to give back
    recorder = Recorder(B._calls)
    monkeypatch.setattr(B, "_calls", recorder)
    assert run(False, wk=w[1], rope=rope) is None and recorder.answers == [("paged_append", None)]


@DTYPES
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("prefix", [0, 20])
def test_attention(monkeypatch, dtype, ragged, prefix):
    g = torch.Generator(device="cuda").manual_seed(3)
    kp, vp = (torch.randn((6, 2, 16, 64), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((6, 4, 64), generator=g, device="cuda").to(dtype)
    table = torch.tensor([[3, 0], [5, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([9, 30], dtype=torch.int32, device="cuda")
    pages = torch.tensor([2, 4], dtype=torch.int32, device="cuda") if prefix else None
    cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda") if ragged else None
    for kw in (dict(), dict(max_q=5), dict(max_len=30), dict(scale=0.3), dict(max_q=4, max_len=32, scale=1.0, lse=True),
               dict(out=torch.empty_like(q))):
        short(monkeypatch, "prefix_attention", lambda: B.prefix_attention(q, kp, vp, table, lens, pages, prefix, cu, **kw))


def test_what_is_written():
    """Behind the table's row, before its begin and on pages outside the pool: exactly the
    rows that have a place are written, and nothing else of the pools."""
    k = torch.ones((12, 1, 64), device="cuda")
    kp, vp = (torch.zeros((6, 1, 4, 64), device="cuda") for _ in range(2))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([0, 6], [1, 2], [3, 4], [-1, 5])  # (page 6 is not there, nor is page -1)
    past = i32(2, 7, -2, 1)
    B.paged_append(None, k, 2 * k, kp, vp, table, past)
    torch.cuda.synchronize()
    rows = {(0, 2), (0, 3), (2, 3), (3, 0)}  # 2, 3 and not 4; 7 and not 8, 9; not -2, -1, but 0; none of 1 .. 3
    for pool, value in ((kp, 1.0), (vp, 2.0)):
        full = (pool[:, 0] == value).all(-1)
        assert {tuple(x) for x in full.nonzero().tolist()} == rows and not pool[:, 0][~full].any()
