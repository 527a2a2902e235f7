"""The microscaled 4-bit operators: storage (quantise, read back) and the grouped expert product.

Storage is exact and compared bit for bit with the definition.  Products are compared with it in 64
bits, within the rounding errors of their fp32 sums (counted in mx4_reference.experts) and one rounding
to the output's type.  Refusals need no GPU."""
import ctypes as C

import numpy as np
import pytest

import mx4_reference as ref
import bit_quantized_moe_router_amd as moe

torch = pytest.importorskip("torch")
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
KINDS = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "mx4": moe.MOE_MX4}


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


# ---- the definition itself -----------------------------------------------------------------------


def test_reference_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :8] = [6, -6, 5, 2.5, 0.25, 0.75, 7.9, -0.1]  # amax 7.9: scale 2^(2-2) = 1
    x[0, 32:36] = [1, 0.125, 0.3, -0.0]                # amax 1: scale 2^-2; 4, 0.5, 1.2, -0
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127, 125]]
    assert ref.dequantize(codes, scales)[0, :8].tolist() == [6, -6, 4, 2, 0, 1, 6, 0]
    assert ref.dequantize(codes, scales)[0, 32:36].tolist() == [1, 0.125, 0.25, 0]
    assert codes[0, 0] == 0xF7 and codes[0, 17] >> 4 == 8  # 6, -6; the zero's sign is kept


# ---- refusals (no device is touched) ----------------------------------------------------------------


def status(name, *args):
    return getattr(moe.lib(), name)(*args)


P = 0x10000  # a non-null, aligned address that is never read


@pytest.mark.parametrize("change,want", [
    (dict(type=2), 1), (dict(type=-1), 1), (dict(rows=-1), 1), (dict(cols=0), 2), (dict(cols=48), 2),
    (dict(cols=(1 << 24) + 32), 2), (dict(rows=1 << 42), 2), (dict(ld=63), 1), (dict(wide=None), 1),
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(codes=P + 8), 1), (dict(wide=P + 2), 1),
])
def test_storage_refusals(change, want):
    a = dict(wide=P, type=0, rows=4, cols=64, ld=64, codes=P, scales=P)
    a.update(change)
    assert status("moe_mx4_quantize", a["wide"], a["type"], a["rows"], a["cols"], a["ld"], a["codes"], a["scales"],
                  None) == want
    assert status("moe_mx4_dequantize", a["codes"], a["scales"], a["rows"], a["cols"], a["wide"], a["type"], a["ld"],
                  None) == want
    assert moe.lib().moe_last_error()


def test_no_rows_is_a_no_op():
    assert status("moe_mx4_quantize", None, 0, 0, 64, 64, None, None, None) == 0
    assert status("moe_mx4_dequantize", None, None, 0, 64, None, 1, 64, None) == 0
    d = moe.make_mx4_desc(4, 64, 64, moe.MOE_BF16, moe.MOE_F32)
    assert status("moe_mx4_experts", C.byref(d), None, None, None, None, 0, None, 0, None, 1, None, None, None, None,
                  0, None) == 0


@pytest.mark.parametrize("desc,change,want", [
    (dict(n_experts=0), {}, 2), (dict(n_experts=513), {}, 2), (dict(k=0), {}, 2), (dict(k=40), {}, 2),
    (dict(k=65568), {}, 2), (dict(n=0), {}, 2), (dict(n=65537), {}, 2), (dict(x_type=0), {}, 1), (dict(x_type=3), {}, 1),
    (dict(y_type=3), {}, 1), (dict(y_type=-1), {}, 1), (dict(swiglu=2), {}, 1), (dict(n=63, swiglu=1), {}, 2),
    (dict(n=48, y_type=2), {}, 2), (dict(n=96, y_type=2, swiglu=1), {}, 2),
    ({}, dict(rows=-1), 1), ({}, dict(rows=(1 << 24) + 1), 1), ({}, dict(x_rows=0), 1), ({}, dict(y_rows=0), 1),
    ({}, dict(src_div=0), 1), ({}, dict(wc=None), 1), ({}, dict(ws=None), 1), ({}, dict(x=None), 1),
    ({}, dict(off=None), 1), ({}, dict(y=None), 1), (dict(x_type=2), dict(xs=None), 1),
    (dict(y_type=2), dict(ys=None), 1), ({}, dict(x_rows=7), 1), ({}, dict(y_rows=7), 1), ({}, dict(wc=P + 4), 1),
    ({}, dict(x=P + 8), 1), ({}, dict(y=P + 2), 1), (dict(y_type=2), dict(y=P + 4), 1),
])
def test_experts_refusals(desc, change, want):
    d = dict(n_experts=4, n=64, k=64, x_type=1, y_type=0, swiglu=0)
    d.update(desc)
    a = dict(wc=P, ws=P, x=P, xs=P, x_rows=8, off=P, rows=8, src=None, src_div=1, dst=None, scale=None, y=P, ys=P,
             y_rows=8)
    a.update(change)
    md = moe.Mx4Desc(*(d[n] for n, _ in moe.Mx4Desc._fields_))
    assert status("moe_mx4_experts", C.byref(md), *a.values(), None) == want
    assert status("moe_mx4_experts", None, *a.values(), None) == 1


def test_binding_checks_tensors():
    x = torch.zeros(4, 64)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for args in ((x, c, s),                                   # not on a GPU
                 (x[:, :40], c, s), (x.double(), c, s), (x.t(), c, s), (x[0], c, s), (x, c[:3], s), (x, c, s.int()),
                 (x, c[:, ::2], s), (x[:1].expand(4, 64), c, s)):
        with pytest.raises(moe.MoEError):
            moe.moe_mx4_quantize(*args)
    w, ws = torch.zeros(2, 8, 32, dtype=torch.uint8), torch.zeros(2, 8, 2, dtype=torch.uint8)
    off, y = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8)
    d = moe.make_mx4_desc(2, 8, 64, moe.MOE_BF16, moe.MOE_F32)
    xb = x.bfloat16()
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.moe_mx4_experts(d, w, ws, xb, None, off, 4, y)
    idx = torch.zeros(4, dtype=torch.int32)
    for kw in (dict(w_codes=w[:1]), dict(w_scales=ws.int()), dict(x=x), dict(x=xb[:, :32]), dict(x_scales=s),
               dict(expert_offsets=off.long()), dict(expert_offsets=off[:2]), dict(y=y.bfloat16()), dict(y=y[:, :7]),
               dict(y_scales=s), dict(src_rows=idx[:3]), dict(dst_rows=idx.long()), dict(row_scale=torch.ones(3))):
        a = dict(w_codes=w, w_scales=ws, x=xb, x_scales=None, expert_offsets=off, rows=4, y=y)
        a.update(kw)
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_mx4_experts(d, **a)
        assert "GPU" not in str(ei.value), kw


def test_kernel_name_before_any_call():
    import threading

    names = []
    t = threading.Thread(target=lambda: names.append(moe.moe_mx4_experts_kernel()))
    t.start()
    t.join()
    assert names == [""]


def test_binding_checks_layouts():
    """A matrix with its rows along another dimension has as many elements, and is refused; flat ones are taken."""
    z = lambda *shape: torch.zeros(*shape, dtype=torch.uint8)  # noqa: E731
    x, c, s = torch.zeros(4, 128), z(4, 64), z(4, 4)
    for call, args in ((moe.moe_mx4_quantize, (x, z(64, 4), s)), (moe.moe_mx4_quantize, (x, c, z(2, 8))),
                       (moe.moe_mx4_dequantize, (z(64, 4), s, x)), (moe.moe_mx4_dequantize, (c, z(8, 2), x))):
        with pytest.raises(moe.MoEError, match="codes|scales"):
            call(*args)
    off = torch.zeros(3, dtype=torch.int32)
    d = moe.make_mx4_desc(2, 96, 128, moe.MOE_MX4, moe.MOE_MX4)
    good = dict(w_codes=z(2, 96, 64), w_scales=z(2, 96, 4), x=z(5, 64), x_scales=z(5, 4), expert_offsets=off, rows=5,
                y=z(5, 48), y_scales=z(5, 3))
    for kw in (dict(w_codes=z(2, 64, 96)), dict(w_codes=z(64, 192)), dict(w_scales=z(2, 4, 96)), dict(w_scales=z(4, 192)),
               dict(x_scales=z(4, 5)), dict(y_scales=z(3, 5))):
        with pytest.raises(moe.MoEError, match=next(iter(kw))):
            moe.moe_mx4_experts(d, **{**good, **kw})
    for kw in ({}, dict(w_codes=z(192, 64), w_scales=z(192, 4)), dict(w_codes=z(2 * 96 * 64), x_scales=z(20))):
        with pytest.raises(moe.MoEError, match="GPU"):
            moe.moe_mx4_experts(d, **{**good, **kw})


def test_binding_refuses_what_32_bits_do_not_hold():
    """Sizes reach the library as 32-bit numbers: none is cut to its low bits.  Tensors without memory."""
    far = 1 << 32
    for at in range(3):
        with pytest.raises(moe.MoEError, match="32 bits"):
            moe.make_mx4_desc(*(far + v if i == at else v for i, v in enumerate((2, 96, 128))), moe.MOE_MX4, moe.MOE_MX4)
    z = lambda *shape: torch.empty(*shape, dtype=torch.uint8, device="meta")  # noqa: E731
    f = lambda *shape, t=torch.int32: torch.empty(*shape, dtype=t, device="meta")  # noqa: E731
    d = moe.make_mx4_desc(2, 32, 32, moe.MOE_MX4, moe.MOE_MX4)
    good = dict(w_codes=z(2, 32, 16), w_scales=z(2, 32, 1), x=z(5, 16), x_scales=z(5, 1), expert_offsets=f(3), rows=5,
                y=z(5, 16), y_scales=z(5, 1))
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.moe_mx4_experts(d, **good)
    for kw in (dict(rows=far + 5), dict(rows=far + 5, src_rows=f(far + 5)), dict(rows=far + 5, dst_rows=f(far + 5)),
               dict(src_div=far + 1), dict(src_div=-far + 1), dict(x=z(far + 5, 16), x_scales=z(far + 5, 1)),
               dict(y=z(far + 5, 16), y_scales=z(far + 5, 1))):
        with pytest.raises(moe.MoEError, match="32 bits"):
            moe.moe_mx4_experts(d, **{**good, **kw})


# ---- storage -------------------------------------------------------------------------------------------


def spread(rows, cols, seed):
    """Values of every magnitude: rows scaled from subnormal to near the largest, ties and zeros among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x = np.ldexp(x, rng.integers(-148, 124, (rows, 1))).astype(np.float32)
    ties = rng.random((rows, cols)) < 0.3
    x = np.where(ties, np.ldexp(rng.integers(-32, 33, (rows, cols)) / 4.0, rng.integers(-130, 120, (rows, 1))), x)
    x = np.where(rng.random((rows, cols)) < 0.1, np.float32(-0.0), x).astype(np.float32)
    x[rows // 2] = 0
    return x


def quantized(x, gpu):
    rows, cols = x.shape
    codes = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device=gpu)
    scales = torch.full((rows, cols // 32), 0xEE, dtype=torch.uint8, device=gpu)
    moe.moe_mx4_quantize(x, codes, scales)
    return codes, scales


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (64, 256), (17, 2048), (257, 160), (5, 8192)])
def test_storage(gpu, rows, cols, dtype):
    x = torch.from_numpy(spread(rows, cols, rows + cols)).to(dtype)
    codes, scales = quantized(x.to(gpu), gpu)
    want_c, want_s = ref.quantize(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    for out in (torch.float32, torch.bfloat16):
        y = torch.full((rows, cols), 7.0, dtype=out, device=gpu)
        moe.moe_mx4_dequantize(codes, scales, y)
        want = torch.from_numpy(ref.dequantize(want_c, want_s)).to(out)  # exact in both types
        assert torch.equal(y.cpu(), want) and torch.equal(y.cpu().signbit(), want.signbit())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_storage_strided_rows(gpu, dtype):
    """Rows inside a wider, misaligned buffer; what lies between them stays."""
    buf = torch.from_numpy(spread(9, 101, 5)).to(dtype).to(gpu)
    x = buf[:, 3:99]
    codes, scales = quantized(x, gpu)
    want = ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
    y = torch.full((9, 101), 7.0, dtype=dtype, device=gpu)
    moe.moe_mx4_dequantize(codes, scales, y[:, 3:99])
    assert torch.equal(y[:, 3:99].double().cpu(), torch.from_numpy(ref.dequantize(*want)))
    assert (y[:, :3] == 7).all() and (y[:, 99:] == 7).all()


@pytest.mark.gpu
def test_storage_nan_and_infinity(gpu):
    x = torch.ones(4, 96)
    x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), -float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        codes, scales = quantized(x.to(dtype).to(gpu), gpu)
        want_c, want_s = ref.quantize(x.numpy())
        assert np.array_equal(scales.cpu().numpy(), want_s) and np.array_equal(codes.cpu().numpy(), want_c)
        y = torch.zeros(4, 96, dtype=dtype, device=gpu)
        moe.moe_mx4_dequantize(codes, scales, y)
        nan = np.repeat(want_s == 255, 32, 1)
        assert np.array_equal(y.isnan().cpu().numpy(), nan) and (y.float().cpu().numpy()[~nan] == 1).all()


@pytest.mark.gpu
def test_read_back_of_every_code_and_scale(gpu):
    scales = torch.arange(255, dtype=torch.uint8).view(255, 1)
    codes = torch.arange(256, dtype=torch.uint8).view(1, 256)[:, [17 * i for i in range(16)]].expand(255, 16).contiguous()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref.dequantize(codes.numpy(), scales.numpy()))
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.empty(255, 32, dtype=dtype, device=gpu)
        moe.moe_mx4_dequantize(codes.to(gpu), scales.to(gpu), y)
        assert torch.equal(y.cpu(), want.to(dtype))


@pytest.mark.gpu
def test_storage_offsets_past_32_bits(gpu):
    """Two rows 2^32 values apart."""
    buf = torch.empty((1 << 32) + 64, dtype=torch.bfloat16, device=gpu)
    x = buf.as_strided((2, 64), (1 << 32, 1))
    x.copy_(torch.from_numpy(spread(2, 64, 3)))
    codes, scales = quantized(x, gpu)
    want = ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
    x.fill_(0)
    moe.moe_mx4_dequantize(codes, scales, x)
    assert torch.equal(x.double().cpu(), torch.from_numpy(ref.dequantize(*want)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_storage_of_more_than_the_caches_hold(gpu, dtype):
    """256 MB of values and more, a few rows of every kind over and over: equal rows give equal codes."""
    few = torch.from_numpy(spread(64, 2048, 6)).to(dtype)
    x = few.to(gpu).repeat(2048, 1)
    codes, scales = quantized(x, gpu)
    want_c, want_s = (torch.from_numpy(a).to(gpu) for a in ref.quantize(few.float().numpy()))
    assert (codes.view(2048, 64, -1) == want_c).all() and (scales.view(2048, 64, -1) == want_s).all()
    y = torch.full_like(x, 7.0)
    moe.moe_mx4_dequantize(codes, scales, y)
    want = torch.from_numpy(ref.dequantize(want_c.cpu().numpy(), want_s.cpu().numpy())).to(dtype).to(gpu)
    assert (y.view(2048, 64, -1) == want).all()


# ---- the expert product ------------------------------------------------------------------------------------


class Experts:
    """Weights [E, n, k] by their codes, read back an expert at a time."""

    def __init__(self, codes, scales, E):
        self.codes, self.scales = codes.reshape(E, -1, codes.shape[-1]), scales.reshape(E, -1, scales.shape[-1])

    def __getitem__(self, e):
        return ref.dequantize(self.codes[e], self.scales[e])


class Product:
    """Weights, rows and routing of one call, on the CPU and the GPU."""

    def __init__(self, gpu, counts, n, k, x_kind, seed, x_rows=None, src=None, src_div=1, dst=None, y_rows=None,
                 row_scale=False, slack=0, random_codes=False):
        rng = np.random.default_rng(seed)
        E = len(counts)
        self.E, self.n, self.k, self.x_kind = E, n, k, x_kind
        self.offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
        self.used = int(self.offsets[-1])
        self.rows = self.used + slack  # positions behind the last expert's range belong to nobody
        self.x_rows = x_rows or self.rows
        self.y_rows = y_rows or self.rows
        if random_codes:
            self.wc = rng.integers(0, 256, (E * n, k // 2), np.uint8)
            self.ws = rng.integers(118, 126, (E * n, k // 32), np.uint8)
        else:
            self.wc, self.ws = ref.quantize((rng.standard_normal((E * n, k)) * 0.05).astype(np.float32))
        self.w = Experts(self.wc, self.ws, E)
        x = torch.from_numpy((rng.standard_normal((self.x_rows, k)) * np.exp(rng.standard_normal((self.x_rows, 1)))
                              ).astype(np.float32)).bfloat16()
        self.src, self.src_div, self.dst = src, src_div, dst
        self.scale = rng.uniform(-1, 1, self.y_rows).astype(np.float32) if row_scale else None
        t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(gpu)  # noqa: E731
        if x_kind == "mx4":
            xc, xs = ref.quantize(x.float().numpy())
            self.x, self.gx, self.gxs = ref.dequantize(xc, xs), t(xc), t(xs)
        else:
            self.x, self.gx, self.gxs = x.double().numpy(), x.to(gpu), None
        self.gwc, self.gws = t(self.wc), t(self.ws)
        self.goff = t(self.offsets)
        self.gsrc, self.gdst = (t(None if a is None else np.asarray(a, np.int32)) for a in (src, dst))
        self.gscale = t(self.scale)
        self.gpu = gpu

    def want(self, swiglu):
        pos = np.arange(self.rows)
        s = pos if self.src is None else np.where(np.asarray(self.src) < 0, -1, np.asarray(self.src) // self.src_div)
        d = pos if self.dst is None else np.asarray(self.dst)
        return ref.experts(self.w, self.x, self.offsets, s, d, self.scale, self.y_rows, swiglu)

    def outputs(self, y_kind, swiglu):
        cols = self.n // 2 if swiglu else self.n
        if y_kind == "mx4":
            return (torch.full((self.y_rows, cols // 2), 0xEE, dtype=torch.uint8, device=self.gpu),
                    torch.full((self.y_rows, cols // 32), 0xEE, dtype=torch.uint8, device=self.gpu))
        dtype = torch.float32 if y_kind == "f32" else torch.bfloat16
        return torch.full((self.y_rows, cols), 7.0, dtype=dtype, device=self.gpu), None

    def call(self, y, ys, y_kind, swiglu):
        d = moe.make_mx4_desc(self.E, self.n, self.k, KINDS[self.x_kind], KINDS[y_kind], swiglu)
        moe.moe_mx4_experts(d, self.gwc, self.gws, self.gx, self.gxs, self.goff, self.rows, y, ys, src_rows=self.gsrc,
                            src_div=self.src_div, dst_rows=self.gdst, row_scale=self.gscale)

    def run(self, y_kind, swiglu):
        y, ys = self.outputs(y_kind, swiglu)
        self.call(y, ys, y_kind, swiglu)
        return (y, ys) if y_kind == "mx4" else y

    def check(self, swiglu, kinds=("f32", "bf16")):
        want, err = self.want(swiglu)
        written = ~np.isnan(want).all(1)
        for kind in kinds:
            y = self.run(kind, swiglu)
            got = y.double().cpu().numpy()
            assert (got[~written] == 7).all(), kind
            # One rounding of a value that is itself err off.
            tol = err + U[y.dtype] * (np.abs(want) + err) + 1e-37
            far = np.abs(got - want)[written] - tol[written]
            assert np.isfinite(got[written]).all() and far.max(initial=-1) <= 0, (kind, far.max())
        cols = want.shape[1]
        if cols % 32 == 0:
            # The codes are those of the fp32 values of the same call.
            codes, scales = (t.cpu().numpy() for t in self.run("mx4", swiglu))
            z = self.run("f32", swiglu).cpu().numpy()
            want_c, want_s = ref.quantize(z)
            assert np.array_equal(codes[written], want_c[written]) and np.array_equal(scales[written], want_s[written])
            assert (codes[~written] == 0xEE).all() and (scales[~written] == 0xEE).all()


# Positions an expert: none, one, and numbers around the tiles' edges.
COUNTS = [[1], [0, 3, 0, 1], [15, 16, 17, 0, 33], [31, 0, 64, 65], [130], [127, 1, 128, 0, 2], [300, 7]]


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("n,k", [(64, 32), (192, 96), (128, 288), (256, 512)])
def test_experts(gpu, counts, n, k, x_kind, swiglu):
    Product(gpu, counts, n, k, x_kind, n + k + len(counts)).check(swiglu)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("n,swiglu", [(1, 0), (2, 1), (31, 0), (33, 0), (70, 1), (130, 0), (1000, 0), (514, 1)])
def test_experts_odd_columns(gpu, n, swiglu, x_kind):
    Product(gpu, [5, 0, 40, 140], n, 160, x_kind, n).check(swiglu)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("tokens", [1, 2, 7, 64, 333])
def test_experts_gather_and_scatter(gpu, tokens, x_kind):
    """Routing as moe_route gives it: rows gathered by token, rows scattered by assignment, weighted."""
    rng = np.random.default_rng(tokens)
    E, k = 12, 3
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(tokens)]).reshape(-1)
    order = np.argsort(ids, kind="stable")
    counts = np.bincount(ids, minlength=E)
    Product(gpu, counts, 192, 256, x_kind, 1, x_rows=tokens, src=order, src_div=k).check(1)
    Product(gpu, counts, 96, 256, x_kind, 2, dst=order, row_scale=True).check(0)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("big", [0, 1])
def test_experts_rows_outside(gpu, x_kind, big):
    """Sources outside x are zero rows, targets outside y and positions behind the last range are not written."""
    counts = [3, 0, 5, 2] if not big else [70, 0, 150, 2]
    rows = sum(counts) + 6
    src = np.arange(rows) % 9
    src[[0, 4, 7]] = [-1, 9, 1 << 30]
    dst = np.arange(rows)[::-1].copy() + 3
    dst[[1, 5]] = [-7, rows + 40]
    p = Product(gpu, counts, 64, 128, x_kind, 3, x_rows=9, src=src, dst=dst, y_rows=rows + 5, row_scale=True, slack=6)
    p.check(0)
    y = p.run("f32", 0)
    assert (y[dst[0]] == 0).all() and (y[dst[4]] == 0).all()


@pytest.mark.gpu
def test_experts_offsets_are_held_inside(gpu):
    """Offsets beyond the arrays or decreasing reach no memory outside them; valid ranges stay right."""
    p = Product(gpu, [4, 4, 4], 64, 64, "bf16", 4)
    want, err = p.want(0)
    p.goff = torch.tensor([0, 4, 2, 1 << 30], dtype=torch.int32, device=gpu)
    y = p.run("f32", 0).double().cpu().numpy()
    assert (np.abs(y[:2] - want[:2]) <= err[:2] + 1e-6 * np.abs(want[:2])).all()
    p.goff = torch.tensor([-5, -5, 900, 1], dtype=torch.int32, device=gpu)
    p.run("f32", 0)
    p.goff = torch.zeros(4, dtype=torch.int32, device=gpu)
    assert (p.run("f32", 0) == 7).all()


def around(E, rows, seed):
    """Counts of E experts, `rows` on average, some of them none."""
    c = np.random.default_rng(seed).integers(0, 2 * rows + 1, E)
    c[E // 3] = 0
    return c


# Sizes large enough for the kernels with tiles of their own shapes: experts' positions, n, k.  k that is no multiple
# of 512, down to a single block, takes their forms for odd lengths.
TILED = [
    ("mx4", [150, 0, 1, 300, 129, 400], 4098, 512),   # 256 x 128
    ("mx4", around(300, 30, 1), 256, 512),            # several tiles of one unit a workgroup
    ("mx4", [700, 3, 1200, 900], 2112, 1536),
    ("mx4", [2050], 4100, 512),                       # 256 x 256
    ("mx4", [4000, 0, 1900, 257, 2500], 2112, 512),
    ("mx4", [1300], 4100, 32),                        # 256 x 128, odd
    ("mx4", [700, 1, 1400, 900], 2112, 288),
    ("mx4", [900, 1, 0, 140], 4098, 544),
    ("bf16", [200], 4100, 1024),                      # 256 x 32
    ("bf16", around(64, 8, 2), 4100, 512),
    ("bf16", around(300, 30, 3), 1026, 32),           # the same, odd
    ("bf16", [600, 0, 33, 300], 4098, 160),
    ("bf16", [4100], 258, 512),                       # 128 x 128
    ("bf16", [500, 0, 1, 129, 1400], 1056, 1024),
    ("bf16", around(40, 70, 4), 1058, 512),           # 256 x 128
    ("bf16", [2100], 2112, 1536),
    ("bf16", [300, 0, 1, 640], 4224, 32),             # the same, odd
    ("bf16", [1500, 130, 1700], 2050, 544),
]


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("x_kind,counts,n,k", TILED, ids=[f"{x}-{len(c)}x{sum(c)}-{n}-{k}" for x, c, n, k in TILED])
def test_experts_tiled(gpu, x_kind, counts, n, k, swiglu):
    Product(gpu, counts, n, k, x_kind, n + k, random_codes=True).check(swiglu)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind,counts,n,k", [
    ("mx4", around(12, 170, 5), 2112, 512), ("mx4", around(6, 1100, 6), 2112, 512), ("mx4", around(12, 300, 7), 2112, 288),
    ("bf16", around(64, 9, 8), 4160, 512), ("bf16", around(4, 500, 9), 4160, 160), ("bf16", around(6, 150, 10), 2112, 1024),
    ("bf16", around(40, 70, 11), 2112, 512), ("bf16", around(6, 900, 12), 2112, 288)])
def test_experts_tiled_gather_and_scatter(gpu, x_kind, counts, n, k):
    """Sources by token, targets by assignment, factors, rows outside on either side and behind the last range."""
    rng = np.random.default_rng(n + k + len(counts))
    rows = int(sum(counts)) + 9
    tokens = (rows + 2) // 3
    src = rng.permutation(3 * tokens)[:rows]
    src[rng.integers(0, rows, 20)] = rng.choice([-1, 3 * tokens, 1 << 30, -(1 << 31)], 20)
    dst = rng.permutation(rows + 7)[:rows]
    dst[rng.choice(rows, 20, replace=False)] = rng.choice([-1, rows + 7, 1 << 30, -(1 << 31)], 20)
    p = Product(gpu, counts, n, k, x_kind, 13, x_rows=tokens, src=src, src_div=3, dst=dst, y_rows=rows + 7, row_scale=True,
                slack=9, random_codes=True)
    p.check(1)
    p.check(0)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind,rows,n,k", [("mx4", 1000, 2112, 512), ("mx4", 2304, 4100, 512), ("bf16", 200, 4100, 1024),
                                             ("bf16", 1024, 2112, 512), ("bf16", 2304, 2112, 1536)])
def test_experts_tiled_unaligned(gpu, x_kind, rows, n, k):
    """Scales and results that begin at no multiple of 16 bytes."""
    p = Product(gpu, [rows // 2, rows - rows // 2], n, k, x_kind, 14, random_codes=True)

    def moved(t, by):
        buf = torch.empty(t.numel() + by, dtype=t.dtype, device=gpu)
        buf[by:].copy_(t.reshape(-1))
        return buf[by:].view(t.shape)

    want, err = p.want(0)
    aligned = p.run("f32", 0)
    y = moved(p.outputs("f32", 0)[0], 1)
    p.call(y, None, "f32", 0)
    assert torch.equal(y, aligned)
    p.gws = moved(p.gws, 1)
    if x_kind == "mx4":
        p.gxs = moved(p.gxs, 2)
    p.call(y, None, "f32", 0)
    assert (np.abs(y.double().cpu().numpy() - want) <= err + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind,rows,n,k", [("mx4", 1000, 2112, 512), ("mx4", 2304, 4100, 512), ("mx4", 2304, 4100, 96),
                                             ("bf16", 200, 4100, 1024), ("bf16", 1024, 2112, 512), ("bf16", 2304, 2112, 1536),
                                             ("bf16", 900, 4100, 96)])
def test_experts_tiled_nan_stays_in_its_row(gpu, x_kind, rows, n, k):
    p = Product(gpu, [rows], n, k, x_kind, 15, random_codes=True)
    clean = p.run("f32", 0)
    if x_kind == "mx4":
        p.gxs[1, 2] = 255
    else:
        p.gx[1, 70] = float("nan")
    p.gws[5, 1] = 255  # a weight block: its column in every row
    y = p.run("f32", 0)
    rest, cols = torch.arange(rows, device=gpu) != 1, torch.arange(n, device=gpu) != 5
    assert y[1].isnan().all() and y[:, 5].isnan().all()
    assert torch.equal(y[rest][:, cols], clean[rest][:, cols])


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
def test_experts_tiled_offsets_are_held_inside(gpu, x_kind):
    """Offsets that rise and fall or lie outside reach no memory outside the arrays."""
    p = Product(gpu, [500] * 6, 2112, 512, x_kind, 16, random_codes=True)
    p.run("f32", 0)
    for off in ([0, 3000, 0, 3000, 0, 3000, 0], [-5, 1 << 30, 7, 7, -(1 << 31), 900, 1], [3000] * 7, [0] * 7):
        p.goff = torch.tensor(off, dtype=torch.int32, device=gpu)
        y = p.run("f32", 0)
        assert y.isfinite().all()
        if off[0] == off[-1]:
            assert off[1] != off[0] or (y == 7).all()


def shifted(t, by):
    """A copy of t that begins `by` elements into its memory."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    buf[by:].copy_(t.reshape(-1))
    return buf[by:].view(t.shape)


# Each kernel: what it is taken for, and which one takes the same product where scales begin at no multiple of 16 bytes.
KERNELS = [
    ("few", "few", "bf16", around(100, 4, 104), 1058, 288),
    ("few", "few", "mx4", around(80, 4, 84), 2112, 288),
    ("few split", "few split", "bf16", [1, 0, 3], 576, 512),
    ("few split", "few split", "mx4", [1, 0, 3], 578, 160),
    ("bf16 256x32", "bf16 256x32 odd", "bf16", around(40, 30, 70), 2112, 512),
    ("bf16 256x32 odd", "bf16 256x32 odd", "bf16", around(40, 30, 70), 2114, 288),
    ("bf16 128x128", "bf16 256x32 odd", "bf16", around(6, 300, 306), 2112, 512),
    ("bf16 128x128", "few", "bf16", around(3, 150, 153), 4864, 512),
    ("bf16 256x128", "bf16 256x128 odd", "bf16", around(12, 150, 162), 2112, 512),
    ("bf16 256x128", "bf16 256x128 odd", "bf16", around(40, 150, 190), 578, 1024),
    ("bf16 256x128 odd", "bf16 256x128 odd", "bf16", around(12, 150, 162), 2114, 160),
    ("4-bit 256x128", "4-bit 256x128 odd", "mx4", around(64, 70, 134), 578, 512),
    ("4-bit 256x128", "few", "mx4", around(6, 300, 306), 2112, 512),
    ("4-bit 256x128 odd", "4-bit 256x128 odd", "mx4", around(40, 70, 110), 2112, 160),
    ("4-bit 256x256", "4-bit 256x128 odd", "mx4", around(12, 300, 312), 2112, 512),
    ("4-bit 256x256", "4-bit 256x128 odd", "mx4", around(64, 150, 214), 578, 512),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,unaligned,x_kind,counts,n,k", KERNELS,
                         ids=[f"{m}-{x}-{sum(c)}-{n}-{k}".replace(" ", "_") for m, _, x, c, n, k in KERNELS])
def test_experts_kernels(gpu, kernel, unaligned, x_kind, counts, n, k):
    """Every kernel by its name, plain; and gathered, scattered and weighted with rows outside on either side, also
    with scales at other addresses, where that takes another kernel."""
    def check(want):
        for swiglu in (0, 1):
            p.check(swiglu)
            # The sizes are chosen for an MI355X's compute units.
            assert moe.moe_mx4_experts_kernel() == want or torch.cuda.get_device_properties(0).multi_processor_count != 256

    p = Product(gpu, counts, n, k, x_kind, n + k, random_codes=True)
    check(kernel)
    rng = np.random.default_rng(n + k + len(counts))
    rows = p.rows + 9
    tokens = (rows + 2) // 3
    src, dst = rng.permutation(3 * tokens)[:rows], rng.permutation(rows + 7)[:rows]
    src[rng.integers(0, rows, 3)] = [-1, 3 * tokens, -(1 << 31)]
    dst[rng.choice(rows, 3, replace=False)] = [-1, rows + 7, 1 << 30]
    p = Product(gpu, counts, n, k, x_kind, 23, x_rows=tokens, src=src, src_div=3, dst=dst, y_rows=rows + 7, row_scale=True,
                slack=9, random_codes=True)
    check(kernel)
    p.gws = shifted(p.gws, 1)
    if x_kind == "mx4":
        p.gxs = shifted(p.gxs, 3)
    check(unaligned)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
def test_experts_many(gpu, x_kind):
    """512 experts with 0 to 9 rows; and all rows with the last expert."""
    rng = np.random.default_rng(8)
    Product(gpu, rng.integers(0, 10, 512), 32, 64, x_kind, 5).check(0)
    Product(gpu, [0] * 511 + [50], 32, 64, x_kind, 6).check(0)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("n,k", [(64, 32), (192, 160), (322, 64)])
def test_experts_many_swiglu(gpu, n, k, x_kind):
    """512 experts with 0 to 9 rows: more tiles than compute units, columns shared out among the waves."""
    rng = np.random.default_rng(n)
    counts = rng.integers(0, 10, 512)
    rows = int(counts.sum())
    Product(gpu, counts, n, k, x_kind, 17, x_rows=rows // 2, src=rng.permutation(rows), src_div=2,
            dst=rng.permutation(rows), row_scale=True).check(1)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("rows", [2, 200])
def test_experts_nan_stays_in_its_row(gpu, x_kind, rows):
    p = Product(gpu, [rows], 64, 128, x_kind, 7)
    clean = p.run("f32", 0)
    if x_kind == "mx4":
        p.gxs[1, 2] = 255
    else:
        p.gx[1, 70] = float("nan")
    y = p.run("f32", 0)
    assert y[1].isnan().all()
    keep = torch.arange(rows) != 1
    assert torch.equal(y[keep], clean[keep])
    p.gws[5, 1] = 255  # a weight block: its column in every row
    y = p.run("f32", 0)
    assert y[:, 5].isnan().all() and not y[keep][:, :5].isnan().any() and not y[keep][:, 6:].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("small", ["w", "x"])
@pytest.mark.parametrize("x_kind,rows,n,k", [("bf16", 3, 64, 96), ("mx4", 3, 64, 96), ("bf16", 200, 4100, 1024),
                                             ("bf16", 1024, 2112, 512), ("bf16", 2304, 2112, 1536), ("bf16", 900, 4100, 96),
                                             ("mx4", 1000, 2112, 512), ("mx4", 2304, 4100, 512), ("mx4", 2304, 4100, 96)])
def test_experts_smallest_and_largest_values(gpu, x_kind, rows, n, k, small):
    """One side near 2^-127, subnormal where it is bf16, the other near 2^115: products of ordinary size, none lost."""
    p = Product(gpu, [rows], n, k, x_kind, 18, random_codes=True)
    rng = np.random.default_rng(19)
    scales = lambda lo, shape: rng.integers(lo, lo + 4, shape).astype(np.uint8)  # noqa: E731
    lo, hi = 0, 240
    p.ws = scales(lo if small == "w" else hi, p.ws.shape)
    p.gws = torch.from_numpy(p.ws).to(gpu)
    p.w = Experts(p.wc, p.ws, 1)
    if x_kind == "mx4":
        xs = scales(hi if small == "w" else lo, (rows, k // 32))
        p.gxs = torch.from_numpy(xs).to(gpu)
        p.x = ref.dequantize(p.gx.cpu().numpy(), xs)
    else:
        bits = rng.integers(1, 0x180, (rows, k)) if small == "x" else rng.integers(0x7780, 0x7900, (rows, k))
        x = torch.from_numpy((bits | rng.integers(0, 2, (rows, k)) << 15).astype(np.int32)).to(torch.int16).view(torch.bfloat16)
        p.gx, p.x = x.to(gpu), x.double().numpy()
    p.check(0)


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("n", [1, 160])
def test_experts_most_rows(gpu, x_kind, n):
    """2^24 positions of a few rows of x, and results past 2^31 values: every row is its source's row of a small call."""
    P_, E, k = 1 << 24, 3, 32
    p = Product(gpu, [7, 7, 7], n, k, x_kind, 22, x_rows=7, src=np.tile(np.arange(7), 3), y_rows=21, random_codes=True)
    table = p.run("f32", 0)  # [expert * 7 + row]
    p.check(0, ("f32",))
    p.goff = torch.tensor([0, 5000001, 5000002, P_], dtype=torch.int32, device=gpu)
    p.rows = p.y_rows = P_
    p.gsrc = torch.arange(P_, dtype=torch.int32, device=gpu) * 5 % 7
    y = p.run("f32", 0)
    step = 1 << 21
    for at in range(0, P_, step):
        i = torch.arange(at, at + step, device=gpu)
        e = (i >= 5000001).long() + (i >= 5000002).long()
        assert torch.equal(y[at:at + step], table[e * 7 + p.gsrc[at:at + step].long()]), at


@pytest.mark.gpu
def test_experts_tiled_in_a_graph(gpu):
    """Large products on two streams of one graph, replayed amid eager calls with other rows."""
    a = Product(gpu, [1300, 0, 1100], 2112, 512, "mx4", 20, random_codes=True)
    b = Product(gpu, [600, 5, 800], 2112, 512, "bf16", 21, random_codes=True)
    outs = [q.outputs("bf16", 0)[0] for q in (a, b)]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        a.call(outs[0], None, "bf16", 0)
        with torch.cuda.stream(side):
            b.call(outs[1], None, "bf16", 0)
        torch.cuda.current_stream().wait_stream(side)
    for turn in range(4):
        a.gx.copy_(a.gx.flip(0))
        b.gx.neg_()
        want = [q.run("bf16", 0) for q in (a, b)]
        for y in outs:
            y.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        assert all(torch.equal(y, w) for y, w in zip(outs, want)), turn


@pytest.mark.gpu
@pytest.mark.parametrize("x_kind", ["bf16", "mx4"])
@pytest.mark.parametrize("rows", [3, 150])
def test_experts_weights_past_32_bits(gpu, x_kind, rows):
    """The last expert's codes start past 2^32 bytes."""
    E, n, k = 512, 4160, 4096
    p = Product(gpu, [rows], n, k, x_kind, 9)
    want, err = p.want(0)
    wc = torch.empty(E, n, k // 2, dtype=torch.uint8, device=gpu)
    ws = torch.empty(E, n, k // 32, dtype=torch.uint8, device=gpu)
    assert (E - 1) * n * (k // 2) > 1 << 32
    wc[-1], ws[-1] = p.gwc, p.gws
    d = moe.make_mx4_desc(E, n, k, KINDS[x_kind], moe.MOE_F32)
    off = torch.zeros(E + 1, dtype=torch.int32, device=gpu)
    off[-1] = rows
    y = torch.empty(rows, n, device=gpu)
    moe.moe_mx4_experts(d, wc, ws, p.gx, p.gxs, off, rows, y)
    assert (np.abs(y.double().cpu().numpy() - want) <= err + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.gpu
def test_experts_repeat_bits_and_streams(gpu):
    """The same bits from call to call, and from two streams at once."""
    a, b = Product(gpu, [40, 3, 0, 90], 256, 512, "mx4", 10), Product(gpu, [1, 1], 256, 512, "bf16", 11)
    ya, yb = a.run("bf16", 1), b.run("bf16", 1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [[], []]
    for _ in range(5):
        for i, p in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                out[i].append(p.run("bf16", 1))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ya) for y in out[0]) and all(torch.equal(y, yb) for y in out[1])


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [2, 300])
def test_layer_chain_in_a_graph(gpu, tokens):
    """Rows quantised, gate/up with SwiGLU into 4 bits, down with the routing weights: the run of an MoE
    layer after moe_route, eager and replayed from a graph with changed rows."""
    import moe_inputs as mi
    from bit_quantized_moe_router_amd.layer import MoELayer, to_dev

    H, E, k, I = 256, 16, 2, 128  # the small layer's sizes
    lay = MoELayer(mi.gen_weights(H, E, I, I, 0), k, device=gpu, max_tokens=512, max_chunk=512)
    rng = np.random.default_rng(tokens)
    gu, gus = (torch.from_numpy(a).to(gpu) for a in ref.quantize(rng.standard_normal((E * 2 * I, H)) * 0.05))
    dn, dns = (torch.from_numpy(a).to(gpu) for a in ref.quantize(rng.standard_normal((E * H, I)) * 0.05))
    P_ = tokens * k
    e8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=gpu)  # noqa: E731
    xc, xs, hc, hs = e8(tokens, H // 2), e8(tokens, H // 32), e8(P_, I // 2), e8(P_, I // 32)
    rows = torch.empty(P_, H, device=gpu)
    x = to_dev(mi.gen_x(tokens, H, 1), gpu)
    d1 = moe.make_mx4_desc(E, 2 * I, H, moe.MOE_MX4, moe.MOE_MX4, 1)
    d2 = moe.make_mx4_desc(E, H, I, moe.MOE_MX4, moe.MOE_F32)
    mt = moe.moe_max_tiles(lay.desc, tokens)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=gpu)  # noqa: E731
    r = dict(topk_ids=i32(tokens, k), topk_weights=torch.zeros(tokens, k, device=gpu), expert_counts=i32(E),
             expert_offsets=i32(E + 1), sorted_assign=i32(P_), tile_map=i32(mt, 3), n_tiles=i32(1))

    def layer():
        moe.moe_route(lay.desc, x, tokens, lay.router_w, None, r, lay.ws)
        moe.moe_mx4_quantize(x.view(torch.bfloat16), xc, xs)
        moe.moe_mx4_experts(d1, gu, gus, xc, xs, r["expert_offsets"], P_, hc, hs, src_rows=r["sorted_assign"], src_div=k)
        moe.moe_mx4_experts(d2, dn, dns, hc, hs, r["expert_offsets"], P_, rows, dst_rows=r["sorted_assign"],
                            row_scale=r["topk_weights"])
        return rows[0::k] + rows[1::k]  # the two assignments of a token

    def reference():
        """From the same codes, in 64 bits; h's own codes from the call, whose rounding the sums cannot repeat."""
        ids, w = r["topk_ids"].cpu().numpy(), r["topk_weights"].double().cpu().numpy()
        order = r["sorted_assign"].cpu().numpy()
        Wd = ref.dequantize(dn.cpu().numpy(), dns.cpu().numpy()).reshape(E, H, I)
        h = np.empty((P_, I))
        h[order] = ref.dequantize(hc.cpu().numpy(), hs.cpu().numpy())
        y = np.zeros((tokens, H))
        for t in range(tokens):
            for j in range(k):
                y[t] += w[t, j] * (Wd[ids[t, j]] @ h[t * k + j])
        return y

    y = layer()
    want = reference()
    # fp32 sums of I products and k rows: far below 1e-5 of the largest value.
    assert np.abs(y.double().cpu().numpy() - want).max() <= 1e-5 * np.abs(want).max()
    xq = ref.dequantize(*ref.quantize(x.view(torch.bfloat16).float().cpu().numpy()))
    assert np.array_equal(ref.dequantize(xc.cpu().numpy(), xs.cpu().numpy()), xq)
    # h against SwiGLU of the exact products: a code is off by at most a quarter of the block's largest value.
    Wg = ref.dequantize(gu.cpu().numpy(), gus.cpu().numpy()).reshape(E, 2 * I, H)
    z = np.stack([Wg[e] @ xq[t] for t, row in enumerate(r["topk_ids"].cpu().numpy()) for e in row])
    hx = z[:, :I] / (1 + np.exp(-z[:, :I])) * z[:, I:]
    h = np.empty((P_, I))
    h[r["sorted_assign"].cpu().numpy()] = ref.dequantize(hc.cpu().numpy(), hs.cpu().numpy())
    block = np.abs(hx).reshape(P_, -1, 32).max(2).repeat(32, 1)
    assert (np.abs(h - hx) <= 0.2501 * block).all()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer()
    for seed in (2, 3, 4):
        x.copy_(to_dev(mi.gen_x(tokens, H, seed), gpu))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, layer()), seed
