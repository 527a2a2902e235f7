"""The combination of routed rows and its gradients, against the definitions in 64 bits of routing_reference.
Refusals need no GPU."""
import numpy as np
import pytest

import routing_reference as ref
import bit_quantized_moe_router_amd as moe

torch = pytest.importorskip("torch")
P = 0x10000  # a non-null, aligned address that is never read
i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


def test_reference_by_hand():
    rows = np.array([[1.0, 2.0], [10.0, 20.0], [np.nan, np.nan], [3.0, 4.0]])
    ids, w = np.array([[0, 1], [-1, 5]]), np.array([[0.5, 0.25], [1.0, 2.0]])
    y, _ = ref.combine(rows, ids, w, np.array([[1.0, 1.0], [0.0, 0.0]]), 2)
    assert y.tolist() == [[4.0, 7.0], [6.0, 8.0]]
    drows, dw, _ = ref.combine_gradient(np.array([[1.0, -1.0], [2.0, 0.0]]), rows, ids, w, 2)
    assert drows.tolist() == [[0.5, -0.5], [0.25, -0.25], [0, 0], [4.0, 0]] and dw.tolist() == [[-1.0, -10.0], [0, 6.0]]


def test_reference_gradient_by_differences():
    rng = np.random.default_rng(0)
    rows, w, dy = rng.standard_normal((6, 5)), rng.standard_normal((2, 3)), rng.standard_normal((2, 5))
    drows, dw, _ = ref.combine_gradient(dy, rows, None, w, 3)
    loss = lambda r, v: (ref.combine(r, None, v, None, 3)[0] * dy).sum()  # noqa: E731
    for i in range(6):
        for j in range(5):
            e = np.zeros((6, 5))
            e[i, j] = 1e-3
            assert abs((loss(rows + e, w) - loss(rows - e, w)) / 2e-3 - drows[i, j]) < 1e-10
    for i in range(2):
        for j in range(3):
            e = np.zeros((2, 3))
            e[i, j] = 1e-3
            assert abs((loss(rows, w + e) - loss(rows, w - e)) / 2e-3 - dw[i, j]) < 1e-10


SHAPE = [(dict(T=-1), 1), (dict(k=0), 1), (dict(k=17), 1), (dict(width=0), 2), (dict(width=(1 << 24) + 1), 2),
         (dict(T=1 << 30), 2), (dict(rows_type=2), 1), (dict(y_type=2), 1), (dict(rows=P + 2), 1)]


@pytest.mark.parametrize("change,want", SHAPE + [
    (dict(rows=None), 1), (dict(y=None), 1), (dict(base=P + 1), 1), (dict(y=P + 2), 1), (dict(T=0, rows=None, y=None), 0)])
def test_forward_refusals(change, want):
    a = dict(rows=P, rows_type=0, T=16, k=4, width=64, ids=None, w=None, base=None, y=P, y_type=0)
    a.update(change)
    assert moe.lib().moe_combine_forward(*a.values(), None) == want


@pytest.mark.parametrize("change,want", SHAPE + [
    (dict(dy=None), 1), (dict(dy=P + 2), 1), (dict(rows=None), 1), (dict(drows=P + 1), 1),
    (dict(drows=None, dw=None), 0), (dict(T=0, rows=None, dy=None), 0)])
def test_backward_refusals(change, want):
    a = dict(dy=P, y_type=0, rows=P, rows_type=0, T=16, k=4, width=64, ids=None, w=None, drows=P, dw=P)
    a.update(change)
    assert moe.lib().moe_combine_backward(*a.values(), None) == want


def test_binding_checks_tensors():
    z = torch.zeros
    good = dict(rows=z(8, 6), topk_ids=z(4, 2, dtype=i32), weights=z(4, 2), base=z(4, 6), y=z(4, 6))
    for kw in (dict(rows=z(7, 6)), dict(rows=z(8, 5)), dict(rows=z(8, 12)[:, ::2]), dict(rows=z(8, 6).half()),
               dict(topk_ids=z(4, 2)), dict(topk_ids=z(2, 4, dtype=i32)), dict(weights=z(4, 3)), dict(weights=z(4, 2).bfloat16()),
               dict(base=z(4, 6).bfloat16()), dict(base=z(3, 6)), dict(y=z(6, 4).t()), dict(y=z(24))):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_combine_forward(**{**good, **kw})
        assert "GPU" not in str(ei.value), kw
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.moe_combine_forward(**good)
    back = dict(dy=z(4, 6), rows=z(8, 6), topk_ids=None, weights=None, drows=z(8, 6), dweights=z(4, 2))
    for kw in (dict(dy=z(4, 5)), dict(drows=z(8, 6).bfloat16()), dict(drows=z(4, 12)), dict(dweights=z(4, 3)),
               dict(rows=None, drows=None), dict(dy=z(4, 6).double())):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_combine_backward(**{**back, **kw})
        assert "GPU" not in str(ei.value), kw
    with pytest.raises(moe.MoEError, match="null"):  # the weights' gradient is made of the rows
        moe._check(moe.lib().moe_combine_backward(P, 0, None, 0, 4, 2, 6, None, None, P, P, None))


# ---- on the GPU ------------------------------------------------------------------------------------------


def half_step(v, dtype):
    """Half a step of the result's type."""
    return (2.0 ** -8 if dtype is bf16 else ref.U) * np.abs(v) + 1e-38


class Combine:
    def __init__(self, gpu, T, k, H, kind, out, seed, base=True, ids=True, weights=True, dropped=0.0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.k = k
        self.rows = r(T * k, H).to(kind).to(gpu)
        self.ids = None
        if ids:
            self.ids = torch.randint(0, 300, (T, k), generator=g, dtype=i32)
            self.ids[torch.rand(T, k, generator=g) < dropped] = -1
            if dropped and T > 2:
                self.ids[T // 2] = -1
            self.ids = self.ids.to(gpu)
        self.w = r(T, k).to(gpu) if weights else None
        self.base = r(T, H).to(out).to(gpu) if base else None
        self.dy = r(T, H).to(out).to(gpu)
        self.y = torch.full((T, H), 9.0, dtype=out, device=gpu)
        self.drows = torch.full_like(self.rows, 9.0)
        self.dw = torch.full((T, k), 9.0, device=gpu)

    def forward(self):
        moe.moe_combine_forward(self.rows, self.ids, self.w, self.base, self.y)

    def backward(self):
        moe.moe_combine_backward(self.dy, self.rows, self.ids, self.w, self.drows, self.dw)

    def outputs(self):
        return [self.y, self.drows, self.dw]

    def check(self):
        n = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        rows, ids, w, base, dy = n(self.rows), n(self.ids), n(self.w), n(self.base), n(self.dy)
        self.forward()
        self.backward()
        y, tol = ref.combine(rows, ids, w, base, self.k)
        assert (np.abs(n(self.y) - y) <= tol + half_step(np.abs(y) + tol, self.y.dtype)).all()
        drows, dw, dtol = ref.combine_gradient(dy, rows, ids, w, self.k)
        # One product in float32, rounded once more to the rows' type.
        assert (np.abs(n(self.drows) - drows) <= half_step(drows, f32) + half_step(drows * (1 + ref.U), self.rows.dtype)).all()
        assert (np.abs(n(self.dw) - dw) <= dtol + 1e-38).all()
        return self


SHAPES = [(1, 8, 2048), (1, 1, 1), (3, 2, 7), (5, 16, 17), (33, 6, 130), (64, 8, 512), (17, 9, 1999), (130, 3, 4099),
          (1030, 8, 96), (1025, 4, 1001), (2085, 2, 30), (2, 5, 70001)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,out", [(f32, f32), (bf16, bf16), (bf16, f32), (f32, bf16)])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_sums_and_gradients(gpu, T, k, H, kind, out):
    Combine(gpu, T, k, H, kind, out, T + H).check()
    Combine(gpu, T, k, H, kind, out, T + H, base=False, dropped=0.3).check()
    Combine(gpu, T, k, H, kind, out, T + H, ids=False, weights=False, base=False).check()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(4, 64), (1500, 40), (40, 3000)])
def test_left_out_rows_may_hold_anything(gpu, T, H):
    """NaN and infinity in rows without an expert, and in their weights, reach nothing; a token without experts is its
    base, or zeros."""
    x = Combine(gpu, T, 4, H, bf16, f32, 1, dropped=0.4)
    gone = x.ids.flatten() < 0
    x.rows[gone] = float("nan")
    x.w.view(-1)[gone] = float("inf")
    y = Combine(gpu, T, 4, H, bf16, f32, 1, dropped=0.4)
    x.forward(), x.backward(), y.forward(), y.backward()
    for a, b in zip(x.outputs(), y.outputs()):
        assert torch.equal(a, b)
    x.ids.fill_(-1)
    x.forward(), x.backward()
    assert torch.equal(x.y, x.base) and not x.drows.any() and not x.dw.any()
    x.base = None
    x.forward()
    assert not x.y.any()


@pytest.mark.gpu
def test_nan_is_not_hidden(gpu):
    x = Combine(gpu, 50, 4, 100, bf16, bf16, 2)
    x.rows[13, 7] = float("nan")
    x.rows[22, 9] = float("inf")
    x.forward(), x.backward()
    assert x.y[3, 7].isnan() and x.y[5, 9].isinf() and int((~x.y.isfinite()).sum()) == 2
    assert x.dw[3, 1].isnan() and int((~x.dw.isfinite()).sum()) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(30, 513), (1100, 513)])
def test_in_place_and_one_output_alone(gpu, T, H):
    x = Combine(gpu, T, 6, H, bf16, bf16, 3, dropped=0.2).check()
    y, drows, dw = (t.clone() for t in x.outputs())
    only = torch.full_like(x.drows, 5.0)
    moe.moe_combine_backward(x.dy, None, x.ids, x.w, only, None)
    assert torch.equal(only, drows)
    other = torch.full_like(x.dw, 5.0)
    moe.moe_combine_backward(x.dy, x.rows, x.ids, x.w, None, other)
    assert torch.equal(other, dw)
    x.y = x.base
    x.forward()
    assert torch.equal(x.y, y)
    x.drows = x.rows
    x.backward()
    assert torch.equal(x.drows, drows) and torch.equal(x.dw, dw)


@pytest.mark.gpu
def test_unaligned_and_nothing(gpu):
    for kind in (f32, bf16):
        x = Combine(gpu, 40, 3, 77, kind, kind, 4, dropped=0.1)
        for name in ("rows", "ids", "w", "base", "dy", "y", "drows", "dw"):
            t = getattr(x, name)
            odd = torch.empty(t.numel() + 1, dtype=t.dtype, device=gpu)[1:].view(t.shape)
            odd.copy_(t)
            setattr(x, name, odd)
        x.check()
        Combine(gpu, 0, 3, 77, kind, kind, 4).forward()
    # What lies behind the last row stays as it was.
    x = Combine(gpu, 5, 3, 13, bf16, bf16, 5)
    room = torch.full((6 * 13,), 4.0, dtype=bf16, device=gpu)
    x.y = room[:65].view(5, 13)
    x.check()
    assert (room[65:] == 4).all()


@pytest.mark.gpu
def test_repeat_bits_streams_and_graph(gpu):
    xs = [Combine(gpu, 700, 8, 1000, bf16, f32, 5, dropped=0.1), Combine(gpu, 1500, 4, 200, f32, bf16, 6)]
    wants = []
    for x in xs:
        x.forward(), x.backward()
        wants.append([t.clone() for t in x.outputs()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                x.forward(), x.backward()
    torch.cuda.synchronize()
    for x, want in zip(xs, wants):
        assert all(torch.equal(t, w) for t, w in zip(x.outputs(), want))
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        for x in xs:
            x.forward(), x.backward()
    for seed in (9, 10, 11):
        ys = [Combine(gpu, 700, 8, 1000, bf16, f32, seed, dropped=0.1), Combine(gpu, 1500, 4, 200, f32, bf16, seed)]
        for x, y in zip(xs, ys):
            for name in ("rows", "ids", "w", "base", "dy"):
                getattr(x, name).copy_(getattr(y, name))
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(xs, ys):
            y.forward(), y.backward()
            assert all(torch.equal(a, b) for a, b in zip(x.outputs(), y.outputs()))


@pytest.mark.gpu
def test_past_32_bits(gpu):
    """More than 2^31 values of rows, the last token's among them."""
    T, k, H = 33000, 16, 4100
    rows = torch.zeros(T * k, H, dtype=bf16, device=gpu)
    rows[-k:] = torch.arange(k, device=gpu, dtype=bf16)[:, None]
    y = torch.full((T, H), 9.0, dtype=bf16, device=gpu)
    moe.moe_combine_forward(rows, None, None, None, y)
    assert (y[-1] == 120).all() and not y[:-1].any()
    dy = torch.zeros(T, H, dtype=bf16, device=gpu)
    dy[-1] = 1
    dw = torch.full((T, k), 9.0, device=gpu)
    moe.moe_combine_backward(dy, rows, None, None, rows, dw)
    assert torch.equal(dw[-1], H * torch.arange(k, device=gpu, dtype=f32)) and not dw[:-1].any()
    assert (rows[-k:] == 1).all() and not rows[:-k].any()
