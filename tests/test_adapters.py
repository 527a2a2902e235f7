"""Low-rank adapters and their gradients against the definitions in 64 bits of routing_reference, and a run of the
operators together.  Refusals need no GPU."""
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
    a, b = np.array([[[1.0, 2.0]], [[0.0, 1.0]]]), np.array([[[3.0], [1.0]], [[-1.0], [2.0]]])
    x = np.array([[1.0, 1.0], [2.0, 0.5]])
    o = ref.adapters(a, b, np.array([2.0, 1.0]), x, [0, 1, 3], np.array([2, 1, 9]), 2, np.array([1, 0, 2]),
                     np.ones((4, 2)), 4, dy=np.eye(4, 2))
    # Position 0: adapter 0, x[1], h = 3; positions 1, 2: adapter 1, x[0] with h = 1 and nothing.
    assert o["h"][0].tolist() == [[3.0], [1.0], [0.0]]
    assert np.array_equal(o["y"][0], [[0, 3], [19, 7], [1, 1], [np.nan] * 2], equal_nan=True)
    # dh_0 = 2 B_0^T (0, 1) = 2; dh_1 = B_1^T (1, 0) = -1.
    assert o["dx"][0][2].tolist() == [2.0, 4.0] and o["dx"][0][1].tolist() == [0.0, -1.0] and np.isnan(o["dx"][0][[0, 3]]).all()
    assert o["da"][0].tolist() == [[[4.0, 1.0]], [[-1.0, -1.0]]] and o["db"][0].tolist() == [[[0.0], [6.0]], [[1.0], [0.0]]]


def test_reference_gradient_by_differences():
    rng = np.random.default_rng(3)
    r = rng.standard_normal
    a, b, s, x, dy = r((2, 2, 3)), r((2, 4, 2)), r(2), r((5, 3)), r((5, 4))
    src = dst = np.arange(5)
    f = lambda a, b, x: (ref.adapters(a, b, s, x, [0, 2, 5], src, 1, dst, None, 5)["y"][0] * dy).sum()  # noqa: E731
    o = ref.adapters(a, b, s, x, [0, 2, 5], src, 1, dst, None, 5, dy=dy)
    for name, which in (("da", 0), ("db", 1), ("dx", 2)):
        t = [a, b, x]
        for at in np.ndindex(t[which].shape):
            v = []
            for step in (1e-3, -1e-3):
                u = [m.copy() for m in t]
                u[which][at] += step
                v.append(f(*u))
            assert abs((v[0] - v[1]) / 2e-3 - o[name][0][at]) < 1e-9


DESC = dict(n=4, r=8, K=64, N=64, y=0)
SHAPE = [(dict(n=0), 2), (dict(n=513), 2), (dict(r=0), 2), (dict(r=129), 2), (dict(K=0), 2), (dict(K=65537), 2), (dict(N=0), 2),
         (dict(N=65537), 2), (dict(y=2), 1)]
ROWS = [(dict(rows=-1), 1), (dict(rows=(1 << 24) + 1), 1), (dict(x_rows=0), 1), (dict(y_rows=0), 1), (dict(src_div=0), 1),
        (dict(a=None), 1), (dict(b=None), 1), (dict(x=None), 1), (dict(offsets=None), 1), (dict(a=P + 1), 1), (dict(x=P + 1), 1),
        (dict(src=None, x_rows=15), 1), (dict(dst=None, y_rows=15), 1)]


def _split(change):
    d = {**DESC, **{k: v for k, v in change.items() if k in DESC}}
    return moe.AdapterDesc(*d.values()), {k: v for k, v in change.items() if k not in DESC}


@pytest.mark.parametrize("change,want", SHAPE + ROWS + [
    (dict(out=None), 1), (dict(out=P + 2), 1), (dict(base=P + 1), 1), (dict(rows=0, a=None, b=None, x=None, out=None), 0)])
def test_forward_refusals(change, want):
    d, change = _split(change)
    a = dict(a=P, b=P, scales=None, x=P, x_rows=16, offsets=P, rows=16, src=P, src_div=1, dst=P, base=None, out=P, y_rows=16,
             h=None)
    a.update(change)
    assert moe.lib().moe_adapters_forward(d, *a.values(), None) == want


@pytest.mark.parametrize("change,want", SHAPE + ROWS + [
    (dict(h=None), 1), (dict(dy=None), 1), (dict(dy=P + 2), 1), (dict(base=P + 1), 1), (dict(dx=P + 1), 1), (dict(da=None), 1),
    (dict(db=None), 1), (dict(dx=None, base=P), 1), (dict(ws=None), 1), (dict(ws=P + 8), 1), (dict(bytes=64), 3),
    (dict(dx=None, da=None, db=None), 0), (dict(rows=0, da=None, db=None, x=None), 0), (dict(rows=0, offsets=None), 1)])
def test_backward_refusals(change, want):
    d, change = _split(change)
    a = dict(a=P, b=P, scales=None, x=P, x_rows=16, h=P, dy=P, y_rows=16, offsets=P, rows=16, src=P, src_div=1, dst=P, base=None,
             dx=P, da=P, db=P, ws=P, bytes=1 << 20)
    a.update(change)
    assert moe.lib().moe_adapters_backward(d, *a.values(), None) == want


def test_null_descriptor_and_workspace_size():
    L = moe.lib()
    assert L.moe_adapters_forward(None, P, P, None, P, 16, P, 16, P, 1, P, None, P, 16, None, None) == 1
    d = moe.make_adapter_desc(4, 16, 64, 64, moe.MOE_F32)
    assert moe.moe_adapters_workspace_bytes(d, 1000) >= 64000
    for bad in (-1, 1 << 25, 1 << 32):
        with pytest.raises(moe.MoEError):
            moe.moe_adapters_workspace_bytes(d, bad)
    with pytest.raises(moe.MoEError, match="32 bits"):
        moe.make_adapter_desc(4, 16, 1 << 33, 64, moe.MOE_F32)


def test_binding_checks_tensors():
    z = torch.zeros
    h = lambda *s: z(*s, dtype=bf16)  # noqa: E731
    i = lambda n: z(n, dtype=i32)  # noqa: E731
    d = moe.make_adapter_desc(3, 4, 10, 6, moe.MOE_F32)
    good = dict(a=h(3, 4, 10), b=h(3, 6, 4), scales=z(3), x=h(5, 10), offsets=i(4), rows=10, base=z(10, 6), y=z(10, 6), h=z(10, 4),
                src_rows=i(10), src_div=2, dst_rows=i(10))
    bad = (dict(a=h(3, 10, 4)), dict(a=z(3, 4, 10)), dict(b=h(3, 4, 6)), dict(b=h(2, 6, 4)), dict(scales=z(4)), dict(x=h(5, 9)),
           dict(x=z(5, 10)), dict(x=h(10, 5).t()), dict(offsets=i(3)), dict(src_rows=i(9)), dict(dst_rows=i(11)),
           dict(src_rows=z(10)))
    for kw in bad + (dict(base=h(10, 6)), dict(base=z(9, 6)), dict(y=h(10, 6)), dict(y=z(10, 7)), dict(h=z(9, 4)), dict(h=h(10, 4))):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_adapters_forward(d, **{**good, **kw})
        assert "GPU" not in str(ei.value), kw
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.moe_adapters_forward(d, **good)
    back = dict(a=good["a"], b=good["b"], scales=None, x=good["x"], h=z(10, 4), dy=z(10, 6), offsets=i(4), rows=10,
                base=h(10, 10), dx=h(10, 10), da=z(3, 4, 10), db=z(3, 6, 4), ws=z(4096, dtype=torch.uint8), src_rows=i(10),
                src_div=2, dst_rows=i(10))
    for kw in bad + (dict(h=z(4, 10)), dict(dy=h(10, 6)), dict(base=h(5, 10)), dict(dx=h(5, 10)), dict(dx=z(10, 10)),
                     dict(da=h(3, 4, 10)), dict(da=z(3, 10, 4)), dict(db=z(3, 4, 6)), dict(ws=z(4096))):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_adapters_backward(d, **{**back, **kw})
        assert "GPU" not in str(ei.value), kw


# ---- on the GPU ------------------------------------------------------------------------------------------


def half_step(v, dtype):
    return (2.0 ** -8 if dtype is bf16 else ref.U) * np.abs(v) + 1e-38


class Adapters:
    """Rows of `lens` positions for each adapter; top_k positions a row of x, gathered, or rows in their order."""

    def __init__(self, gpu, lens, r, K, N, out, seed, top_k=1, gather=True, base=True, scales=True, extra=0):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        n, rows = len(lens), int(sum(lens))
        if top_k > 1:
            rows = (rows + top_k - 1) // top_k * top_k
        self.n, self.rows, self.top_k, self.out = n, rows + extra, top_k, out
        T = rows // top_k
        self.desc = moe.make_adapter_desc(n, r, K, N, moe.MOE_F32 if out is f32 else moe.MOE_BF16)
        self.offsets = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=i32).to(gpu)
        places = torch.randperm(rows, generator=g).to(i32) if gather else None
        # Positions behind the last adapter's name rows as well: they must have no effect.
        self.places = None if places is None else torch.cat((places, torch.zeros(extra, dtype=i32))).to(gpu)
        self.a, self.b = (rn(n, r, K) / K ** 0.5).to(bf16).to(gpu), (0.3 * rn(n, N, r)).to(bf16).to(gpu)
        self.scales = (torch.rand(n, generator=g) + 0.5).to(gpu) if scales else None
        self.x = rn(T + (0 if gather else extra), K).to(bf16).to(gpu)
        y_rows = rows + extra
        self.base = rn(y_rows, N).to(out).to(gpu) if base else None
        self.dy = rn(y_rows, N).to(out).to(gpu)
        self.y = torch.full((y_rows, N), 9.0, dtype=out, device=gpu)
        self.h = torch.full((self.rows, r), 9.0, device=gpu)
        self.dx_base = rn(len(self.x) * (top_k if gather else 1), K).to(bf16).to(gpu) if base else None
        self.dx = torch.full((len(self.x) * (top_k if gather else 1), K), 9.0, dtype=bf16, device=gpu)
        self.da, self.db = torch.full((n, r, K), 9.0, device=gpu), torch.full((n, N, r), 9.0, device=gpu)
        self.ws = torch.full((moe.moe_adapters_workspace_bytes(self.desc, self.rows),), 0xEE, dtype=torch.uint8, device=gpu)

    def kw(self):
        return dict(src_rows=self.places, src_div=self.top_k, dst_rows=self.places)

    def forward(self):
        moe.moe_adapters_forward(self.desc, self.a, self.b, self.scales, self.x, self.offsets, self.rows, self.base, self.y,
                                 self.h, **self.kw())

    def backward(self):
        moe.moe_adapters_backward(self.desc, self.a, self.b, self.scales, self.x, self.h, self.dy, self.offsets, self.rows,
                                  self.dx_base, self.dx, self.da, self.db, self.ws, **self.kw())

    def outputs(self):
        return [self.y, self.h, self.dx, self.da, self.db]

    def inputs(self):
        return [self.a, self.b, self.x, self.dy] + [t for t in (self.base, self.dx_base, self.scales, self.places) if t is not None]

    def check(self):
        n = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        base, dx_base = n(self.base), n(self.dx_base)
        self.forward()
        self.backward()
        off = self.offsets.cpu().numpy()
        places = np.arange(self.rows) if self.places is None else self.places.cpu().numpy()
        s = np.ones(self.n) if self.scales is None else n(self.scales)
        o = ref.adapters(n(self.a), n(self.b), s, n(self.x), off, places, self.top_k, places, base, len(self.y), n(self.dy),
                         self.out is f32)
        if dx_base is not None:
            o["dx"][0] += dx_base
            o["dx"][1] += ref.U * np.abs(o["dx"][0])
        for name in ("y", "h", "dx", "da", "db"):
            want, tol = o[name]
            got = n(getattr(self, name))
            there = ~np.isnan(want)
            assert (got[~there] == 9).all(), name  # nothing written where no position is
            far = np.abs(got - want)[there] - (tol + half_step(np.abs(want) + tol, getattr(self, name).dtype))[there]
            assert far.max(initial=-1) <= 0, (name, far.max())
        return self


# Lengths by adapter, rank, widths.
CASES = [([1], 16, 64, 64), ([3, 0, 5], 8, 32, 40), ([0, 0, 17, 1], 16, 128, 256), ([40, 7], 4, 100, 60), ([33], 24, 72, 200),
         ([16, 16, 1], 32, 264, 136), ([5, 70, 0, 130], 64, 200, 72), ([9, 21], 128, 160, 96), ([12], 1, 1, 1), ([7, 2], 3, 13, 9),
         ([20, 50], 50, 77, 131), ([31, 0, 2], 100, 65, 33), ([400, 90], 16, 520, 1032), ([257], 12, 1000, 48), ([1] * 70, 16, 96, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("out", [f32, bf16])
@pytest.mark.parametrize("lens,r,K,N", CASES)
def test_rows_and_gradients(gpu, lens, r, K, N, out):
    Adapters(gpu, lens, r, K, N, out, r + K).check()
    Adapters(gpu, lens, r, K, N, out, r + K, gather=False, base=False, scales=False, extra=3).check()


@pytest.mark.gpu
@pytest.mark.parametrize("out", [f32, bf16])
def test_gathered_rows(gpu, out):
    """Several positions a row of x, as routed rows have them, and positions behind the last adapter's."""
    Adapters(gpu, [10, 0, 22, 64, 4], 16, 128, 192, out, 1, top_k=4).check()
    Adapters(gpu, [100, 20, 6], 40, 136, 88, out, 2, top_k=3, extra=9).check()


@pytest.mark.gpu
@pytest.mark.parametrize("r", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("out", [f32, bf16])
def test_many_rows(gpu, r, out):
    """The tiles of several blocks of 16 rows."""
    rng = np.random.default_rng(r)
    cuts = np.sort(rng.integers(0, 17000, 5))
    lens = np.diff(np.concatenate(([0], cuts, [17000]))).tolist()
    Adapters(gpu, lens, r, 128, 72, out, r, extra=5).check()


@pytest.mark.gpu
@pytest.mark.parametrize("out", [f32, bf16])
@pytest.mark.parametrize("n,r,K,N", [(40, 16, 520, 264), (40, 40, 523, 257), (48, 64, 512, 136), (20, 100, 648, 272),
                                     (190, 16, 512, 256), (190, 30, 516, 250), (140, 64, 640, 384), (90, 128, 704, 520)])
def test_many_adapters(gpu, n, r, K, N, out):
    """Columns enough for each of the weight gradients' workgroups, adapters with no row, with few and with many."""
    rng = np.random.default_rng(n + r)
    lens = rng.integers(0, 6, n)
    lens[[1, n // 2, n - 1]] = 0, 300, 70
    Adapters(gpu, lens.tolist(), r, K, N, out, n, extra=3).check()


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(24, 16), (25, 17)])
def test_rows_outside(gpu, K, N):
    """Source rows outside x count as zeros; destinations outside y are not written; bad offsets reach nothing."""
    x = Adapters(gpu, [20, 30], 8, K, N, f32, 5, base=False)
    p = x.places.clone()
    p[3], p[17], p[30] = -1, 50, 1 << 30
    x.places = p
    x.check()
    room = torch.full((60, N), 7.0, device=gpu)
    for off in ([0, 90, 50], [-5, 20, 1 << 30], [40, 10, 50], [50, 50, 50]):
        x.offsets = torch.tensor(off, dtype=i32, device=gpu)
        x.y = room[5:55]
        x.forward()
        x.backward()
        assert (room[:5] == 7).all() and (room[55:] == 7).all()


@pytest.mark.gpu
def test_masked_rows_may_hold_anything(gpu):
    """NaN in rows of x, dy and base that no position names, and in h behind the last position."""
    for rows in (40, 17000):
        x = Adapters(gpu, [rows // 2, 0, rows // 4], 16, 40, 24, f32, 6, extra=rows // 4)
        want = [t.clone() for t in (x.check(), x)[1].outputs()]
        named = torch.zeros(len(x.x), dtype=torch.bool, device=gpu)
        named[x.places[:int(x.offsets[-1])].long()] = True
        for t in (x.x, x.dx_base):
            t[~named[:len(t)]] = float("nan")
        behind = torch.ones(len(x.y), dtype=torch.bool, device=gpu)
        behind[x.places[:int(x.offsets[-1])].long()] = False
        x.base[behind] = float("nan")
        x.dy[behind] = float("nan")
        x.forward()
        x.h[int(x.offsets[-1]):] = float("nan")
        x.backward()
        for a, b in zip([x.y, x.dx, x.da, x.db], [want[0], want[2], want[3], want[4]]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_nan_and_infinity_stay_in_their_row(gpu):
    for bad in (float("nan"), float("inf")):
        x = Adapters(gpu, [20, 30], 16, 64, 64, f32, 7)
        row = int(x.places[5])
        x.x[row, 3] = bad
        x.forward()
        gone = ~x.y.isfinite()
        assert gone[row].all() and int(gone.sum()) == 64
        x = Adapters(gpu, [20, 30], 16, 64, 64, f32, 7)
        x.dy[row, 3] = bad
        x.forward()
        x.backward()
        gone = ~x.dx.isfinite()
        assert gone[row].all() and int(gone.sum()) == 64
        assert not x.da[0].isfinite().all() and x.da[1].isfinite().all() and x.db[1].isfinite().all()


@pytest.mark.gpu
def test_in_place_and_one_output_alone(gpu):
    for rows in (50, 17000):
        x = Adapters(gpu, [rows - 20, 20], 16, 96, 80, bf16, 8).check()
        y, _, dx, da, db = (t.clone() for t in x.outputs())
        x.dx.fill_(9.0)
        a = [x.desc, x.a, x.b, x.scales, x.x, x.h, x.dy, x.offsets, x.rows]
        moe.moe_adapters_backward(*a, x.dx_base, x.dx, None, None, None, **x.kw())
        assert torch.equal(x.dx, dx)
        x.da.fill_(9.0), x.db.fill_(9.0)
        moe.moe_adapters_backward(*a, None, None, x.da, x.db, x.ws, **x.kw())
        assert torch.equal(x.da, da) and torch.equal(x.db, db)
        moe.moe_adapters_forward(x.desc, x.a, x.b, x.scales, x.x, x.offsets, x.rows, x.base, x.base, None, **x.kw())
        assert torch.equal(x.base, y)
        moe.moe_adapters_backward(*a, x.dx_base, x.dx_base, None, None, None, **x.kw())
        assert torch.equal(x.dx_base, dx)


@pytest.mark.gpu
def test_no_rows(gpu):
    x = Adapters(gpu, [0, 0], 16, 96, 80, bf16, 8, gather=False, extra=4)
    x.forward()
    x.backward()
    assert (x.y == 9).all() and (x.h == 9).all() and (x.dx == 9).all() and not x.da.any() and not x.db.any()
    y = Adapters(gpu, [0, 0], 16, 96, 80, bf16, 8)
    y.forward()
    y.backward()
    assert not y.da.any() and not y.db.any()


@pytest.mark.gpu
def test_unaligned_tensors(gpu):
    for out in (f32, bf16):
        x = Adapters(gpu, [20, 45], 16, 64, 72, out, 9)
        for name in ("a", "b", "x", "base", "y", "dy", "h", "dx", "dx_base", "da", "db", "offsets", "places", "scales"):
            t = getattr(x, name)
            odd = torch.empty(t.numel() + 1, dtype=t.dtype, device=gpu)[1:].view(t.shape)
            odd.copy_(t)
            setattr(x, name, odd)
        x.check()


@pytest.mark.gpu
def test_repeat_bits_streams_and_graph(gpu):
    new = lambda s: [Adapters(gpu, [700, 0, 300], 16, 512, 256, bf16, s),  # noqa: E731
                     Adapters(gpu, [1, 1, 0, 2, 64], 32, 128, 264, f32, s + 1, top_k=2)]
    xs = new(5)
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
    for seed in (9, 20, 31):
        ys = new(seed)
        for x, y in zip(xs, ys):
            for t, u in zip(x.inputs(), y.inputs()):
                t.copy_(u)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(xs, ys):
            y.forward(), y.backward()
            assert all(torch.equal(a, b) for a, b in zip(x.outputs(), y.outputs()))


@pytest.mark.gpu
def test_gradient_by_differences(gpu):
    """The float32 output's own slope along a direction of A, of B and of x."""
    x = Adapters(gpu, [30, 40], 8, 64, 48, f32, 12, base=False)
    x.forward()
    x.backward()
    for name, grad in (("a", x.da), ("b", x.db), ("x", x.dx.float())):
        t = getattr(x, name)
        keep = t.clone()
        # y is linear in each of them, so that any step will do: one that bf16 takes exactly.
        way = torch.sign(grad) * 2.0 ** -3
        value = []
        for sign in (1, -1):
            t.copy_((keep.float() + sign * way).to(bf16))
            x.forward()
            value.append((x.y.double() * x.dy).sum())
        taken = ((keep.float() + way).to(bf16).double() - (keep.float() - way).to(bf16).double())
        want = (grad.double() * taken).sum()
        # Float32 sums of 70 x 48 outputs, and dx is rounded to bf16.
        size = float((x.y.double() * x.dy).abs().sum())
        assert abs(float(value[0] - value[1] - want)) <= 2.0 ** -18 * size + 2.0 ** -8 * float((grad.double() * taken).abs().sum())
        t.copy_(keep)


@pytest.mark.gpu
def test_operators_together(gpu):
    """Logits -> experts -> gate/up with an adapter for each expert -> down -> combination, and all the way back to the
    logits, in a graph, against autograd in 64 bits of the same formulas."""
    T, E, k, H, I, r = 96, 16, 4, 128, 64, 8
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = rn(T, H).to(bf16).to(gpu)
    logits = (1.5 * rn(T, E)).to(gpu)
    bias = (0.1 * rn(E)).to(gpu)
    valid = (torch.rand(T, generator=g) < 0.9).to(torch.uint8).to(gpu)

    def stored(*s):
        w = (rn(*s) / s[-1] ** 0.5).to(gpu)
        c = torch.empty(s[0] * s[1], s[2] // 2, dtype=torch.uint8, device=gpu)
        sc = torch.empty(s[0] * s[1], s[2] // 32, dtype=torch.uint8, device=gpu)
        moe.moe_mx4_quantize(w.view(-1, s[2]), c, sc)
        back = torch.empty(s[0] * s[1], s[2], device=gpu)
        moe.moe_mx4_dequantize(c, sc, back)
        return c, sc, back.view(s).double().cpu()

    upc, ups, up = stored(E, I, H)
    dnc, dns, down = stored(E, H, I)
    a, b = (rn(E, r, H) / H ** 0.5).to(bf16).to(gpu), (0.3 * rn(E, I, r)).to(bf16).to(gpu)
    base, dy = rn(T, H).to(gpu), rn(T, H).to(gpu)
    e = lambda *s, t=f32: torch.empty(*s, dtype=t, device=gpu)  # noqa: E731
    sd = moe.make_select_desc(E, k, moe.MOE_SIGMOID, 4, 2, 2, 1, 2.0)
    ad = moe.make_adapter_desc(E, r, H, I, moe.MOE_F32)
    ud = moe.make_mx4_desc(E, I, H, moe.MOE_BF16, moe.MOE_F32)
    dd = moe.make_mx4_desc(E, H, I, moe.MOE_BF16, moe.MOE_F32)
    ids, w, counts, offsets, order = e(T, k, t=i32), e(T, k), e(E, t=i32), e(E + 1, t=i32), e(T * k, t=i32)
    sws = e(moe.moe_select_workspace_bytes(T, E, k), t=torch.uint8)
    aws = e(moe.moe_adapters_workspace_bytes(ad, T * k), t=torch.uint8)
    # Rows of padding tokens' assignments are never written: they hold what they held.
    z, hb, rows, h = torch.zeros(T * k, I, device=gpu), torch.zeros(T * k, I, dtype=bf16, device=gpu), e(T * k, H), e(T * k, r)
    rows.fill_(float("nan"))
    y, drows, dw, dlogits = e(T, H), e(T * k, H), e(T, k), e(T, E)
    dz, dx, dxt = e(T * k, I), torch.zeros(T * k, H, dtype=bf16, device=gpu), e(T, H, t=bf16)
    da, db = e(E, r, H), e(E, I, r)
    place = dict(src_rows=order, src_div=k, dst_rows=order)
    dn32 = down.to(gpu).float()

    def step():
        moe.moe_select_forward(sd, logits, bias, valid, ids, w, counts, offsets, order, sws)
        moe.moe_mx4_experts(ud, upc, ups, x, None, offsets, T * k, z, **place)
        moe.moe_adapters_forward(ad, a, b, None, x, offsets, T * k, z, z, h, **place)
        hb.copy_(z)
        moe.moe_mx4_experts(dd, dnc, dns, hb, None, offsets, T * k, rows, src_rows=order, dst_rows=order)
        moe.moe_combine_forward(rows, ids, w, base, y)
        moe.moe_combine_backward(dy, rows, ids, w, drows, dw)
        # The down product's own gradient by elementary operations.
        torch.sum(drows[:, :, None] * dn32[ids.clamp(min=0).flatten().long()], 1, out=dz)
        moe.moe_adapters_backward(ad, a, b, None, x, h, dz, offsets, T * k, None, dx, da, db, aws, **place)
        moe.moe_combine_forward(dx, ids, None, None, dxt)
        moe.moe_select_backward(sd, logits, ids, w, dw, None, dlogits)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    outs = [ids, w, y, da, db, dxt, dlogits]
    first = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(3):
        for t in outs:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip(outs, first))

    want, _, _ = ref.select(logits.double().cpu().numpy(), k, False, 4, 2, 2, True, 2.0, bias.double().cpu().numpy(),
                            valid.cpu().numpy())
    assert np.array_equal(ids.cpu().numpy(), want)
    A, B, X, L = (t.double().cpu().requires_grad_() for t in (a, b, x, logits))
    total = base.double().cpu().clone()
    on = ids.cpu() >= 0
    at = ids.cpu().clamp(min=0).long()
    sc = torch.sigmoid(L).gather(1, at)
    weights = 2 * sc / sc.sum(1, keepdim=True) * on
    out = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        ex = at[:, j]
        hz = torch.einsum("trh,th->tr", A[ex], X)
        zz = torch.einsum("tih,th->ti", up[ex], X.detach()) + torch.einsum("tir,tr->ti", B[ex], hz)
        row = torch.einsum("thi,ti->th", down[ex], zz)
        out = out + weights[:, j:j + 1] * row
    loss = ((total + out) * dy.double().cpu()).sum()
    loss.backward()
    # The intermediate is rounded to bf16 (2^-8) before the down product, I terms with random signs; dx twice more.
    for got, grad, tol in ((y.double().cpu(), (total + out).detach(), 2.0 ** -8), (da.double().cpu(), A.grad, 2.0 ** -16),
                           (db.double().cpu(), B.grad, 2.0 ** -16), (dxt.double().cpu(), X.grad, 2.0 ** -7),
                           (dlogits.double().cpu(), L.grad, 2.0 ** -7)):
        assert (got - grad).norm() <= tol * grad.norm(), (tol, (got - grad).norm() / grad.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("out", [f32, bf16])
@pytest.mark.parametrize("r,K,N", [(2, 3, 5), (16, 64, 64), (16, 33, 20), (24, 40, 72), (32, 64, 128), (50, 77, 131), (64, 72, 40),
                                   (128, 64, 200)])
def test_numbers_between_hold_24_bits(gpu, r, K, N, out):
    """Whole numbers of 21 bits between the products, in pairs whose differences are the results: exact in every sum."""
    x = Adapters(gpu, [20, 0, 30], r, K, N, out, 13, base=False, scales=False)
    g = torch.Generator().manual_seed(r)

    def wide(rows, cols):
        m = torch.zeros(rows, cols)
        m[:, :3] = torch.randint(0, 128, (rows, 3), generator=g) * torch.tensor([2.0 ** 14, 2.0 ** 7, 1.0])
        return m, m[:, 2:3].double()

    def pairs(cols):  # column c takes one pair's difference
        m = torch.zeros(cols, r)
        pair = 2 * (torch.arange(cols) % (r // 2))
        sign = (torch.randint(0, 2, (cols,), generator=g) * 2 - 1).float()
        m[torch.arange(cols), pair], m[torch.arange(cols), pair + 1] = sign, -sign
        return m, sign.double()

    takes = torch.zeros(r, 3)  # of the even ranks all three numbers, of the odd ones the first two
    takes[:, :2] = 1
    takes[0:r // 2 * 2:2, 2] = 1
    xs, last = wide(len(x.x), K)
    back, sign = pairs(N)
    x.x.copy_(xs)
    x.a.zero_()
    x.a[:, :, :3] = takes.to(bf16).to(gpu)
    x.b.copy_(back.to(bf16).to(gpu).expand_as(x.b))
    x.forward()
    assert torch.equal(x.y.double().cpu(), last * sign)
    dys, last = wide(len(x.dy), N)
    fore, sign = pairs(K)
    x.dy.copy_(dys)
    x.b.zero_()
    x.b[:, :3] = takes.t().to(bf16).to(gpu)
    x.a.copy_(fore.t().to(bf16).to(gpu).expand_as(x.a))
    x.backward()
    assert torch.equal(x.dx.double().cpu(), last * sign)


@pytest.mark.parametrize("where", ["dy", "x", "dy_end", "x_end", "both"])
@pytest.mark.parametrize("gather", [False, True])
def test_overlapping_gradient_is_refused(where, gather):
    """dx over dy, and over x where the factors' gradients read it later; by its last or its first bytes alone too."""
    L, K, N, rows, div = moe.lib(), 24, 40, 16, 2 if gather else 1
    d = moe.make_adapter_desc(4, 8, K, N, moe.MOE_F32)
    x, dy, dx = 1 << 20, 2 << 20, 3 << 20
    x_bytes, dy_bytes, dx_bytes = rows * K * 2, rows * N * 4, rows * div * K * 2
    at = {"dy": dy, "x": x, "dy_end": dy + dy_bytes - 2, "x_end": x - dx_bytes + 2, "both": dy + dy_bytes // 2}[where]

    def call(dx, da):
        return L.moe_adapters_backward(d, P, P, None, x, rows, P, dy, rows, P, rows, P if gather else None, div, None, None, dx,
                                       P if da else None, P if da else None, P, 1 << 20, None)

    assert call(at, True) == 1 and b"overlap" in L.moe_last_error()
    if where not in ("x", "x_end"):
        assert call(at, False) == 1 and b"overlap" in L.moe_last_error()
    if torch.cuda.is_available():
        return  # what is not refused would run
    # Next to them, and over x alone where nothing reads it later: refused for want of a device only.
    for at in (dx, dy + dy_bytes, dy - dx_bytes, x + x_bytes, x - dx_bytes):
        assert call(at, True) != 1
    assert call(x, False) != 1
