"""The router's balance loss, its counts and its gradient, against the definition in 64 bits
(mx4_reference.balance) and against differences.  Refusals need no GPU."""
import numpy as np
import pytest

import mx4_reference as ref
import bit_quantized_moe_router_amd as moe

torch = pytest.importorskip("torch")
P = 0x10000  # a non-null, aligned address that is never read


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


def test_reference_by_hand():
    # Two tokens, two experts, p = (3/4, 1/4) and (1/2, 1/2); both choose expert 0: f = (1, 0), P_0 = 5/8.
    logits = np.array([[np.log(3.0), 0.0], [0.0, 0.0]])
    losses, counts, mean, n, d = ref.balance(logits, np.zeros((2, 1), int), None, 1.0, 0.0)
    assert np.allclose(losses, [2 * 5 / 8, 2 * 5 / 8, (np.log(4.0) ** 2 + np.log(2.0) ** 2) / 2])
    assert counts.tolist() == [2, 0] and np.allclose(mean, [5 / 8, 3 / 8]) and n == 2
    assert np.allclose(d, [[3 / 16, -3 / 16], [1 / 4, -1 / 4]])


def test_reference_gradient_by_differences():
    rng = np.random.default_rng(0)
    logits, ids = rng.standard_normal((6, 5)), rng.integers(0, 5, (6, 2))
    valid = np.array([1, 1, 0, 1, 1, 1])
    d = ref.balance(logits, ids, valid, 0.7, 0.3, 1.5)[4]
    for t in range(6):
        for e in range(5):
            up, down = logits.copy(), logits.copy()
            up[t, e] += 1e-5
            down[t, e] -= 1e-5
            slope = 1.5 * (ref.balance(up, ids, valid, 0.7, 0.3)[0][0] - ref.balance(down, ids, valid, 0.7, 0.3)[0][0]) / 2e-5
            assert abs(slope - d[t, e]) <= 1e-8


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), 1), (dict(E=0), 2), (dict(E=513), 2), (dict(k=0), 1), (dict(k=17), 1), (dict(T=1 << 30), 2),
    (dict(type=2), 1), (dict(logits=None), 1), (dict(logits=P + 2), 1), (dict(ids=None), 1), (dict(losses=None), 1),
    (dict(counts=None), 1), (dict(mean=None), 1), (dict(n=None), 1), (dict(ws=None), 1), (dict(ws=P + 4), 1),
    (dict(bytes=64), 3),
])
def test_forward_refusals(change, want):
    a = dict(logits=P, type=0, T=16, E=8, ids=P, k=2, valid=None, a=0.1, b=0.1, losses=P, counts=P, mean=P, n=P, ws=P,
             bytes=1 << 20)
    a.update(change)
    assert moe.lib().moe_balance_loss_forward(*a.values(), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), 1), (dict(E=0), 2), (dict(E=513), 2), (dict(k=0), 1), (dict(k=17), 1), (dict(type=2), 1),
    (dict(logits=None), 1), (dict(counts=None), 1), (dict(n=None), 1), (dict(dlogits=None), 1),
    (dict(dlogits=P + 2), 1), (dict(T=0, logits=None, counts=None, n=None, dlogits=None), 0),
])
def test_backward_refusals(change, want):
    a = dict(logits=P, type=0, T=16, E=8, k=2, valid=None, a=0.1, b=0.1, counts=P, n=P, grad=None, dlogits=P)
    a.update(change)
    assert moe.lib().moe_balance_loss_backward(*a.values(), None) == want


def test_workspace_size():
    assert 0 < moe.moe_balance_loss_workspace_bytes(0, 1) <= moe.moe_balance_loss_workspace_bytes(65536, 512) < 8 << 20
    for bad in ((-1, 8), (8, 0), (8, 513)):
        with pytest.raises(moe.MoEError):
            moe.moe_balance_loss_workspace_bytes(*bad)


def test_binding_checks_tensors():
    z, i = torch.zeros, torch.int32
    good = dict(logits=z(4, 8), topk_ids=z(4, 2, dtype=i), valid=None, balance_coef=0.1, z_coef=0.1, losses=z(3),
                counts=z(8, dtype=i), mean_prob=z(8), n_valid=z(1, dtype=i), ws=z(1 << 16, dtype=torch.uint8))
    for kw in (dict(logits=z(8, 4).t()), dict(logits=z(4, 8).double()), dict(logits=z(32)), dict(topk_ids=z(3, 2, dtype=i)),
               dict(topk_ids=z(4, 2)), dict(valid=z(4)), dict(valid=z(5, dtype=torch.uint8)), dict(losses=z(2)),
               dict(counts=z(8)), dict(mean_prob=z(9)), dict(n_valid=z(2, dtype=i)), dict(ws=z(8))):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_balance_loss_forward(**{**good, **kw})
        assert "GPU" not in str(ei.value), kw
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.moe_balance_loss_forward(**good)
    back = dict(logits=z(4, 8), top_k=2, valid=None, balance_coef=0.1, z_coef=0.1, counts=z(8, dtype=i),
                n_valid=z(1, dtype=i), grad_loss=None, dlogits=z(4, 8))
    for kw in (dict(dlogits=z(4, 8).bfloat16()), dict(dlogits=z(4, 9)), dict(grad_loss=z(2)), dict(counts=z(7, dtype=i))):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_balance_loss_backward(**{**back, **kw})
        assert "GPU" not in str(ei.value), kw


def test_binding_checks_the_gradients_layout():
    z, i = torch.zeros, torch.int32
    back = dict(logits=z(4, 8), top_k=2, valid=None, balance_coef=0.1, z_coef=0.1, counts=z(8, dtype=i),
                n_valid=z(1, dtype=i), grad_loss=None)
    for shape, match in (((8, 4), "dlogits"), ((2, 16), "dlogits"), ((32,), "GPU"), ((4, 8), "GPU")):
        with pytest.raises(moe.MoEError, match=match):
            moe.moe_balance_loss_backward(dlogits=z(shape), **back)


def test_binding_refuses_what_32_bits_do_not_hold():
    """Sizes reach the library as 32-bit numbers: none is cut to its low bits.  Tensors without memory."""
    T = (1 << 32) + 4
    e = lambda *shape, t=torch.float32: torch.empty(*shape, dtype=t, device="meta")  # noqa: E731
    i = torch.int32
    forward = dict(valid=None, balance_coef=0.1, z_coef=0.1, losses=e(3), n_valid=e(1, t=i), ws=e(1 << 16, t=torch.uint8))
    back = dict(valid=None, balance_coef=0.1, z_coef=0.1, n_valid=e(1, t=i), grad_loss=None)
    for t, E, k in ((T, 1, 1), (4, T, 1), (4, 1, T)):
        with pytest.raises(moe.MoEError, match="32 bits"):
            moe.moe_balance_loss_forward(logits=e(t, E), topk_ids=e(t, k, t=i), counts=e(E, t=i), mean_prob=e(E), **forward)
        with pytest.raises(moe.MoEError, match="32 bits"):
            moe.moe_balance_loss_backward(logits=e(t, E), top_k=k, counts=e(E, t=i), dlogits=e(t, E), **back)
    for bad in ((T, 8), (8, T)):
        with pytest.raises(moe.MoEError, match="32 bits"):
            moe.moe_balance_loss_workspace_bytes(*bad)


# ---- on the GPU ------------------------------------------------------------------------------------------


class Loss:
    def __init__(self, logits, ids, valid, a=0.02, b=0.003):
        self.logits, self.ids, self.valid, self.a, self.b = logits, ids, valid, a, b
        T, E = logits.shape
        dev = logits.device
        self.losses, self.mean = torch.full((3,), 9.0, device=dev), torch.full((E,), 9.0, device=dev)
        self.counts, self.n = (torch.full((m,), -9, dtype=torch.int32, device=dev) for m in (E, 1))
        # A workspace that holds anything at all.
        self.ws = torch.full((moe.moe_balance_loss_workspace_bytes(T, E),), 0xEE, dtype=torch.uint8, device=dev)
        self.d = torch.full_like(logits, 9.0)
        self.grad = torch.tensor([1.25], device=dev)

    def forward(self):
        moe.moe_balance_loss_forward(self.logits, self.ids, self.valid, self.a, self.b, self.losses, self.counts,
                                     self.mean, self.n, self.ws)

    def backward(self, grad=True):
        moe.moe_balance_loss_backward(self.logits, self.ids.shape[1], self.valid, self.a, self.b, self.counts, self.n,
                                      self.grad if grad else None, self.d)

    def check(self):
        self.forward()
        self.backward()
        v = None if self.valid is None else self.valid.cpu().numpy()
        losses, counts, mean, n, d = ref.balance(self.logits.double().cpu().numpy(), self.ids.cpu().numpy(), v, self.a,
                                                 self.b, 1.25)
        T, E = self.logits.shape
        u = 2.0 ** -24
        # A probability: exp's argument is off by |l - top| u, with log2(e) some steps more, the instruction, the
        # sum over E (at most a few steps a tree level) and the division add a few: (16 + 2 range) u, relative.
        span = self.logits.double().cpu()
        span = span.masked_fill(torch.isinf(span), 0)
        span = float((span.amax() - span.amin())) if T else 0.0
        rp = (24 + 4 * span) * u
        # P_e: at most T / (partial rows) fp32 additions of positive numbers; every one has one rounding.
        adds = 64 + T / 64
        got = self.mean.double().cpu().numpy()
        assert np.array_equal(self.counts.cpu().numpy(), counts) and int(self.n) == n
        assert (np.abs(got - mean) <= (rp + adds * u) * mean + 1e-30).all()
        # lse = top + log2(sum) ln 2: a few steps of its largest part, relative to max(|lse|, |top|, log E).
        big = span + float(self.logits.abs().masked_fill(torch.isinf(self.logits), 0).max() if T else 0) + np.log(E) + 1
        rl = 8 * u * big + rp
        gl = self.losses.double().cpu().numpy()
        assert abs(gl[1] - losses[1]) <= (rp + (adds + 2) * u) * losses[1] + 1e-30
        assert abs(gl[2] - losses[2]) <= 2 * rl * big + u * losses[2] + 1e-30
        assert abs(gl[0] - losses[0]) <= self.a * abs(gl[1] - losses[1]) + self.b * abs(gl[2] - losses[2]) + 2 * u * abs(losses[0]) + 1e-30
        # Gradient: p (f - sum + z lse), each factor with its own error.
        p = torch.softmax(self.logits.double().cpu(), 1).nan_to_num(0).numpy()
        f = counts / max(1, n * self.ids.shape[1])
        size = 1.25 * p * (self.a * E / max(1, n) * (f + (p * f).sum(1, keepdims=True)) + 2 * self.b * big / max(1, n))
        tol = size * (2 * rp + 16 * u) + 1.25 * p * 2 * self.b * rl / max(1, n) + 1e-36
        if self.d.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(d) + tol) + 1e-38
        far = np.abs(self.d.double().cpu().numpy() - d) - tol
        assert far.max(initial=-1) <= 0, far.max()


def make(gpu, T, E, k, dtype, seed, masked=0.0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn(T, E, generator=g)).to(dtype)
    ids = torch.topk(logits.float(), k, 1).indices.to(torch.int32) if T else torch.zeros(0, k, dtype=torch.int32)
    valid = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
    return logits.to(gpu), ids.contiguous().to(gpu), None if valid is None else valid.to(gpu)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (2, 7, 3), (63, 8, 2), (64, 16, 2), (129, 33, 4), (500, 100, 5),
                                   (1000, 64, 16), (777, 130, 8), (2085, 256, 8), (300, 511, 16), (4099, 512, 8), (20000, 5, 1)])
def test_loss_and_gradient(gpu, T, E, k, dtype):
    Loss(*make(gpu, T, E, k, dtype, T + E)).check()
    Loss(*make(gpu, T, E, k, dtype, T + E, masked=0.4)).check()


# More than 64 experts (up to 64, up to 32): the forward pass takes workgroups of 1024 threads and 256 partial rows from
# 8192 (16384, 32768) tokens on; from twice as many on a group of lanes goes through more than one row there, as it
# does in the gradient from 16384 (32768, 65536) on.  Rows of each width with 16-byte loads and without.
MANY = [(8193, 100, 4), (16385, 48, 2), (32769, 20, 2), (16390, 256, 8), (33333, 255, 8), (24001, 512, 8), (16389, 511, 16),
        (33001, 128, 2), (17003, 127, 1), (33001, 64, 2), (40001, 63, 5), (70001, 24, 2), (65601, 21, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", MANY)
def test_many_tokens(gpu, T, E, k, dtype):
    Loss(*make(gpu, T, E, k, dtype, T + E, masked=0.3)).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(33001, 100, 4), (70001, 24, 2)])
def test_many_tokens_in_place_repeated_and_on_two_streams(gpu, T, E, k, dtype):
    """Every row is loaded before its gradient replaces it, and bits repeat, also of two calls at once."""
    xs = [Loss(*make(gpu, T, E, k, dtype, seed, masked=0.2)) for seed in (1, 2)]
    wants = []
    for x in xs:
        x.check()
        wants.append([t.clone() for t in (x.losses, x.counts, x.mean, x.d)])
    logits = [x.logits.clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for x, s, l in zip(xs, streams, logits):
            with torch.cuda.stream(s):
                x.logits.copy_(l)
                x.d = x.logits
                x.forward()
                x.backward()
        torch.cuda.synchronize()
        for x, want in zip(xs, wants):
            assert all(torch.equal(t, w) for t, w in zip((x.losses, x.counts, x.mean, x.d), want))


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_many_tokens_nan_stays_in_its_row(gpu, bad):
    """A row that a group of lanes comes to after others, and what it comes to after it."""
    logits, ids, _ = make(gpu, 33001, 100, 2, torch.float32, 3)
    logits[20000, 3] = bad
    x = Loss(logits, ids, None)
    x.forward()
    x.backward()
    assert x.losses.isnan().all() and x.d[20000].isnan().all()
    assert not x.d[:20000].isnan().any() and not x.d[20001:].isnan().any()
    valid = torch.ones(33001, dtype=torch.bool, device=gpu)
    valid[20000] = False
    y = Loss(logits, ids, valid)
    y.forward()
    y.backward()
    assert not y.losses.isnan().any() and not y.d.isnan().any() and not y.d[20000].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 700])
def test_no_valid_token_and_no_token(gpu, T):
    logits, ids, _ = make(gpu, T, 40, 3, torch.float32, 1)
    x = Loss(logits, ids, torch.zeros(T, dtype=torch.bool, device=gpu))
    x.check()
    assert not x.losses.any() and not x.counts.any() and not x.mean.any() and not x.d.any()
    y = Loss(logits[:0], ids[:0], None)
    y.forward()
    y.backward()
    assert not y.losses.any() and not y.counts.any() and not y.mean.any() and int(y.n) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 600])
def test_masked_experts_and_empty_rows(gpu, T):
    """-inf logits, a row of nothing else, ids outside the experts and twice in a row."""
    logits, ids, valid = make(gpu, T, 70, 4, torch.float32, 2, masked=0.2)
    logits[:, 5:9] = -float("inf")
    logits[1] = -float("inf")
    valid[1] = 1
    ids[0] = torch.tensor([-1, 70, 6, 6], dtype=torch.int32)
    ids[2, 1] = 1 << 30
    x = Loss(logits, ids, valid)
    x.check()
    assert not x.d[1].any() and not x.d[:, 5:9].any()


@pytest.mark.gpu
def test_large_logits(gpu):
    """One logit far above the rest, rows far from zero: nothing overflows."""
    logits, ids, _ = make(gpu, 200, 30, 2, torch.float32, 3)
    logits[:, 4] += 80
    logits[::2] -= 3000
    logits[1::2] += 500
    Loss(logits, ids, None).check()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_is_not_hidden(gpu, bad):
    logits, ids, _ = make(gpu, 600, 40, 2, torch.float32, 4)
    logits[7, 3] = bad
    x = Loss(logits, ids, None)
    x.forward()
    x.backward()
    assert x.losses.isnan().all() and x.d[7].isnan().all()
    assert not x.d[:7].isnan().any() and not x.d[8:].isnan().any()
    valid = torch.ones(600, dtype=torch.uint8, device=gpu)
    valid[7] = 0  # in a padding token's row it does not count
    y = Loss(logits, ids, valid)
    y.forward()
    y.backward()
    assert not y.losses.isnan().any() and not y.d.isnan().any() and not y.d[7].any()


@pytest.mark.gpu
def test_gradient_by_differences(gpu):
    """The float32 loss's own slope along a direction."""
    logits, ids, valid = make(gpu, 300, 24, 3, torch.float32, 5, masked=0.1)
    x = Loss(logits, ids, valid, a=1.0, b=0.1)
    x.forward()
    x.backward(grad=False)
    way = torch.sign(x.d)
    h = 0.05
    values = []
    for step in (h, -h):
        y = Loss(logits + step * way, ids, valid, a=1.0, b=0.1)
        y.forward()
        values.append(float(y.losses[0]))
    slope = float((x.d.double() * way).sum())
    # The third derivative's share of a central difference is h^2/6 of it; loss values carry 2^-22 relative.
    assert abs((values[0] - values[1]) / (2 * h) - slope) <= h * h * abs(slope) * 10 + 2.0 ** -22 * abs(values[0]) / h


@pytest.mark.gpu
def test_gradient_in_place_of_the_logits(gpu):
    logits, ids, valid = make(gpu, 500, 200, 4, torch.bfloat16, 6, masked=0.1)
    x = Loss(logits, ids, valid)
    x.forward()
    x.backward()
    want = x.d
    x.d = x.logits
    x.backward()
    assert torch.equal(x.d, want)


@pytest.mark.gpu
def test_repeat_bits_streams_and_graph(gpu):
    """The same bits from call to call, from two streams at once, and from a graph replayed on new logits."""
    xs = [Loss(*make(gpu, 3000, 256, 8, torch.float32, 7, masked=0.1)), Loss(*make(gpu, 900, 512, 4, torch.bfloat16, 8))]
    wants = []
    for x in xs:
        x.forward()
        x.backward()
        wants.append([t.clone() for t in (x.losses, x.counts, x.mean, x.d)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                x.forward()
                x.backward()
    torch.cuda.synchronize()
    for x, want in zip(xs, wants):
        assert all(torch.equal(t, w) for t, w in zip((x.losses, x.counts, x.mean, x.d), want))
    x = xs[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x.forward()
        x.backward()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.forward()
        x.backward()
    for seed in (9, 10, 11):
        logits, ids, _ = make(gpu, 3000, 256, 8, torch.float32, seed)
        x.logits.copy_(logits)
        x.ids.copy_(ids)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (x.losses, x.counts, x.mean, x.d)]
        y = Loss(logits, ids, x.valid)
        y.forward()
        y.backward()
        assert all(torch.equal(t, w) for t, w in zip(got, (y.losses, y.counts, y.mean, y.d)))


@pytest.mark.gpu
def test_with_the_router(gpu):
    """moe_route's choice counted: the counts are its own histogram."""
    import moe_inputs as mi
    from bit_quantized_moe_router_amd.layer import MoELayer, to_dev

    case = mi.make_case("tiny")
    lay = MoELayer(case["w"], case["k"], device=gpu, max_tokens=64)
    x = to_dev(case["x"], gpu)
    r = lay.route(x)
    logits = x.view(torch.bfloat16).float() @ lay.router_w.t()
    loss = Loss(logits.contiguous(), r["topk_ids"], None)
    loss.check()
    assert torch.equal(loss.counts, r["expert_counts"])
