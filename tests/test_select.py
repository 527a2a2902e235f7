"""Routing from scores, the order of assignments by expert, and the logits' gradient, against the definitions in 64
bits of routing_reference and against differences.  Refusals need no GPU."""
import numpy as np
import pytest

import routing_reference as ref
import bit_quantized_moe_router_amd as moe

torch = pytest.importorskip("torch")
P = 0x10000  # a non-null, aligned address that is never read
i32 = torch.int32


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return "cuda"


def test_reference_by_hand():
    # Four experts, scores 1/2, 1/4, 1/8, 1/8: bias lifts the third over the second, ties go left.
    l = np.log(np.array([[4.0, 2.0, 1.0, 1.0]]))
    ids, w, _ = ref.select(l, 2, True, bias=[0, 0, 0.2, 0])
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[0.8, 0.2]])
    ids, w, _ = ref.select(l, 3, True, renorm=False, scale=2.0)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, [[1.0, 0.5, 0.25]])
    # Groups {0, 1} and {2, 3}: by the best 0.5 against 0.6; by the sum of two 0.95 against 0.7.
    l = np.array([[0.0, -np.log(1 / 0.45 - 1), np.log(0.6 / 0.4), np.log(0.1 / 0.9)]])
    assert ref.select(l, 2, False, 2, 1, 1)[0].tolist() == [[2, 3]]
    assert ref.select(l, 2, False, 2, 1, 2)[0].tolist() == [[0, 1]]
    counts, offsets, places = ref.order([[2, 0], [-1, 2], [0, 5]], 3)
    assert counts.tolist() == [2, 0, 2] and offsets.tolist() == [0, 2, 2, 4] and places.tolist() == [1, 4, 0, 3]


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_by_differences(softmax, renorm):
    rng = np.random.default_rng(1)
    l, dw = rng.standard_normal((4, 7)), rng.standard_normal((4, 3))
    ids, w, _ = ref.select(l, 3, softmax, renorm=renorm, scale=1.7)
    d, _ = ref.select_gradient(l, ids, w, dw, softmax, renorm, 1.7)
    for t in range(4):
        for e in range(7):
            v = []
            for step in (1e-6, -1e-6):
                m = l.copy()
                m[t, e] += step
                new, wm, _ = ref.select(m, 3, softmax, renorm=renorm, scale=1.7)
                assert (new == ids).all()
                v.append((wm * dw).sum())
            assert abs((v[0] - v[1]) / 2e-6 - d[t, e]) < 1e-8


DESC = dict(n_experts=8, top_k=2, scores=0, n_groups=1, top_groups=1, group_best=1, renormalise=1, scale=1.0)
BAD_DESC = [(dict(n_experts=0), 2), (dict(n_experts=513), 2), (dict(top_k=0), 1), (dict(top_k=17, n_experts=64), 1),
            (dict(top_k=9), 1), (dict(scores=2), 1), (dict(scores=-1), 1), (dict(n_groups=0), 2), (dict(n_groups=3), 2),
            (dict(n_groups=128, n_experts=128), 2), (dict(n_groups=2, top_groups=3), 1), (dict(top_groups=0), 1),
            (dict(n_groups=4, top_groups=1, top_k=3), 1), (dict(group_best=0), 1), (dict(group_best=3), 1),
            (dict(renormalise=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=0.0), 1)]


@pytest.mark.parametrize("change,want", BAD_DESC)
def test_bad_descriptors(change, want):
    d = moe.SelectDesc(*{**DESC, **change}.values())
    L = moe.lib()
    assert L.moe_select_forward(d, P, 0, 16, None, None, P, P, P, P, P, P, 1 << 20, None) == want
    assert L.moe_select_backward(d, P, 0, 16, P, P, P, None, P, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), 1), (dict(T=1 << 30), 2), (dict(type=2), 1), (dict(logits=None), 1), (dict(logits=P + 2), 1),
    (dict(ids=None), 1), (dict(w=None), 1), (dict(counts=None), 1), (dict(offsets=None), 1), (dict(order=None), 1),
    (dict(ws=None), 1), (dict(ws=P + 8), 1), (dict(bytes=16), 3), (dict(desc=None), 1),
    (dict(T=0, logits=None, ids=None, w=None, counts=None, offsets=None, order=None, ws=None, bytes=0), 0),
])
def test_forward_refusals(change, want):
    a = dict(desc=moe.SelectDesc(*DESC.values()), logits=P, type=0, T=64, bias=None, valid=None, ids=P, w=P, counts=P,
             offsets=P, order=P, ws=P, bytes=1 << 20)
    a.update(change)
    assert moe.lib().moe_select_forward(*a.values(), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), 1), (dict(type=2), 1), (dict(logits=None), 1), (dict(ids=None), 1), (dict(w=None), 1), (dict(dw=None), 1),
    (dict(base=P + 1), 1), (dict(d=None), 1), (dict(d=P + 2), 1), (dict(base=P), 1), (dict(desc=None), 1),
    (dict(T=0, logits=None, ids=None, w=None, dw=None, d=None), 0),
])
def test_backward_refusals(change, want):
    a = dict(desc=moe.SelectDesc(*DESC.values()), logits=P, type=0, T=64, ids=P, w=P, dw=P, base=None, d=P)
    a.update(change)
    assert moe.lib().moe_select_backward(*a.values(), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(n=-1), 1), (dict(E=0), 2), (dict(E=513), 2), (dict(ids=None), 1), (dict(counts=None), 1), (dict(offsets=None), 1),
    (dict(order=None), 1), (dict(ws=None), 1), (dict(ws=P + 4), 1), (dict(bytes=8), 3),
])
def test_sort_refusals(change, want):
    a = dict(ids=P, n=100, E=8, counts=P, offsets=P, order=P, ws=P, bytes=1 << 20)
    a.update(change)
    assert moe.lib().moe_sort_assignments(*a.values(), None) == want


def test_workspace_sizes():
    assert 0 < moe.moe_select_workspace_bytes(0, 1, 1) <= moe.moe_select_workspace_bytes(1 << 20, 512, 16) <= 1 << 20
    assert 0 < moe.moe_sort_workspace_bytes(0, 1) <= moe.moe_sort_workspace_bytes((1 << 31) - 1, 512) <= 1 << 20
    for bad in ((-1, 8, 1), (8, 0, 1), (8, 513, 1), (8, 8, 0), (8, 8, 17), (1 << 30, 8, 4), (1 << 40, 8, 1)):
        with pytest.raises(moe.MoEError):
            moe.moe_select_workspace_bytes(*bad)
    for bad in ((-1, 8), (8, 0), (8, 513), (1 << 31, 8), (8, 1 << 40)):
        with pytest.raises(moe.MoEError):
            moe.moe_sort_workspace_bytes(*bad)
    with pytest.raises(moe.MoEError, match="32 bits"):
        moe.make_select_desc((1 << 32) + 8, 1)


def test_binding_checks_tensors():
    z = torch.zeros
    d = moe.make_select_desc(8, 2)
    good = dict(logits=z(4, 8), bias=None, valid=None, topk_ids=z(4, 2, dtype=i32), topk_weights=z(4, 2),
                expert_counts=z(8, dtype=i32), expert_offsets=z(9, dtype=i32), sorted_assign=z(8, dtype=i32),
                ws=z(1 << 16, dtype=torch.uint8))
    for kw in (dict(logits=z(8, 4).t()), dict(logits=z(4, 9)), dict(logits=z(4, 8).half()), dict(bias=z(7)),
               dict(bias=z(8).bfloat16()), dict(valid=z(4)), dict(valid=z(5, dtype=torch.bool)), dict(topk_ids=z(4, 2)),
               dict(topk_ids=z(2, 4, dtype=i32)), dict(topk_weights=z(4, 3)), dict(expert_counts=z(7, dtype=i32)),
               dict(expert_offsets=z(8, dtype=i32)), dict(sorted_assign=z(9, dtype=i32)), dict(sorted_assign=None),
               dict(expert_counts=None), dict(ws=z(64))):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_select_forward(d, **{**good, **kw})
        assert "GPU" not in str(ei.value), kw
    with pytest.raises(moe.MoEError, match="GPU"):
        moe.moe_select_forward(d, **good)
    back = dict(logits=z(4, 8), topk_ids=z(4, 2, dtype=i32), topk_weights=z(4, 2), dweights=z(4, 2), base=None,
                dlogits=z(4, 8))
    for kw in (dict(dlogits=z(4, 8).bfloat16()), dict(dlogits=z(8, 4)), dict(base=z(4, 7)), dict(base=z(8, 4).t()),
               dict(base=z(4, 8).bfloat16()), dict(dweights=z(4, 3)), dict(dweights=z(2, 4)), dict(topk_ids=z(4, 2))):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_select_backward(d, **{**back, **kw})
        assert "GPU" not in str(ei.value), kw
    sort = dict(ids=z(10, dtype=i32), n_experts=8, expert_counts=z(8, dtype=i32), expert_offsets=z(9, dtype=i32),
                sorted_assign=z(10, dtype=i32), ws=z(1 << 16, dtype=torch.uint8))
    for kw in (dict(ids=z(10)), dict(ids=z(20, dtype=i32)[::2]), dict(sorted_assign=z(9, dtype=i32)),
               dict(expert_offsets=z(8, dtype=i32)), dict(n_experts=7)):
        with pytest.raises(moe.MoEError) as ei:
            moe.moe_sort_assignments(**{**sort, **kw})
        assert "GPU" not in str(ei.value), kw


# ---- on the GPU ------------------------------------------------------------------------------------------


class Select:
    def __init__(self, logits, k, softmax=True, groups=1, top_groups=1, best=1, renorm=True, scale=1.0, bias=None,
                 valid=None, seed=0, base=False):
        T, E = logits.shape
        dev = logits.device
        self.kw = dict(softmax=softmax, groups=groups, top_groups=top_groups, best=best, renorm=renorm, scale=scale)
        self.logits, self.k, self.bias, self.valid = logits, k, bias, valid
        self.desc = moe.make_select_desc(E, k, moe.MOE_SOFTMAX if softmax else moe.MOE_SIGMOID, groups, top_groups, best,
                                         int(renorm), scale)
        full = lambda *s, v=-9, t=i32: torch.full(s, v, dtype=t, device=dev)  # noqa: E731
        self.ids, self.w = full(T, k), full(T, k, v=9.0, t=torch.float32)
        self.counts, self.offsets, self.order = full(E), full(E + 1), full(T * k, v=-7)
        # A workspace that holds anything at all.
        self.ws = full(moe.moe_select_workspace_bytes(T, E, k), v=0xEE, t=torch.uint8)
        g = torch.Generator().manual_seed(seed + 77)
        self.dw = torch.randn(T, k, generator=g).to(dev)
        self.base = torch.randn(T, E, generator=g).to(logits.dtype).to(dev) if base else None
        self.d = torch.full_like(logits, 9.0)

    def forward(self, order=True):
        moe.moe_select_forward(self.desc, self.logits, self.bias, self.valid, self.ids, self.w,
                               *((self.counts, self.offsets, self.order, self.ws) if order else ()))

    def backward(self):
        moe.moe_select_backward(self.desc, self.logits, self.ids, self.w, self.dw, self.base, self.d)

    def outputs(self):
        return [self.ids, self.w, self.counts, self.offsets, self.order, self.d]

    def check(self):
        self.forward()
        self.backward()
        l = self.logits.double().cpu().numpy()
        T, E = l.shape
        bias = None if self.bias is None else self.bias.double().cpu().numpy()
        valid = None if self.valid is None else self.valid.cpu().numpy()
        ids, w, bad = ref.select(l, self.k, bias=bias, valid=valid, **self.kw)
        got = self.w.double().cpu().numpy()
        assert np.array_equal(self.ids.cpu().numpy(), ids)
        finite = np.where(np.isfinite(l), l, 0)
        span = float(finite.max() - finite.min()) if T else 0.0
        # An exponential's argument is off by a rounding of at most the logits' span, with log2(e) some steps more;
        # the instruction, sums and division add a few: relative.
        rel = (24 + 4 * span) * ref.U
        assert (np.isnan(got) == np.isnan(w)).all()
        assert (np.abs(got - w)[~bad] <= rel * np.abs(w[~bad]) + 1e-37).all()
        counts, offsets, order = ref.order(ids, E)
        assert np.array_equal(self.counts.cpu().numpy(), counts) and np.array_equal(self.offsets.cpu().numpy(), offsets)
        places = self.order.cpu().numpy()
        assert np.array_equal(places[:len(order)], order) and (places[len(order):] == -7).all()
        d, size = ref.select_gradient(l, ids, w, self.dw.double().cpu().numpy(), self.kw["softmax"], self.kw["renorm"],
                                      self.kw["scale"])
        base = np.zeros((T, E)) if self.base is None else self.base.double().cpu().numpy()
        have = self.d.double().cpu().numpy()
        tol = (4 * rel + 32 * ref.U) * size + ref.U * np.abs(base) + 1e-36
        if self.logits.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(d + base) + tol)
        else:
            tol = tol + ref.U * np.abs(d + base)
        assert np.isnan(have[bad]).all()
        far = (np.abs(have - (d + base)) - tol)[~bad]
        assert far.max(initial=-1) <= 0, far.max()
        return self


def make(gpu, T, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)).to(dtype)
    return logits.to(gpu), (0.1 * torch.randn(E, generator=g)).to(gpu), (torch.rand(T, generator=g) < 0.8).to(gpu)


SHAPES = [(1, 1, 1), (1, 256, 8), (2, 7, 3), (7, 512, 16), (33, 60, 4), (64, 16, 2), (129, 33, 5), (300, 100, 6),
          (777, 130, 8), (500, 256, 8), (1029, 512, 16), (4099, 24, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_scores(gpu, T, E, k, dtype):
    logits, bias, valid = make(gpu, T, E, dtype, T + E)
    for softmax in (True, False):
        Select(logits, k, softmax).check()
        Select(logits, k, softmax, renorm=False, scale=2.5, bias=bias, valid=valid).check()
        Select(logits, k, softmax, bias=bias, base=True).check()
        Select(logits, k, softmax, renorm=False, valid=valid, base=True).check()


GROUPS = [(5, 32, 4, 2, 8), (66, 256, 8, 4, 8), (100, 60, 3, 1, 4), (50, 512, 64, 3, 16), (70, 64, 64, 9, 6),
          (1300, 96, 4, 2, 10), (40, 35, 7, 6, 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,n,top,k", GROUPS)
def test_groups(gpu, T, E, n, top, k, dtype):
    logits, bias, valid = make(gpu, T, E, dtype, T + E)
    for best in (1, 2):
        for softmax in (True, False):
            # Without a bias, sums of a sigmoid at x and at -x are all 1: such groups are left to the float32 logits.
            if dtype is torch.float32 or softmax or best == 1:
                Select(logits, k, softmax, n, top, best, valid=valid).check()
            Select(logits, k, softmax, n, top, best, bias=bias, renorm=False).check()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("T", [3, 200])
def test_equal_logits(gpu, T, softmax):
    """Ties go to the lower index, of experts and of groups, with a bias and without."""
    g = torch.Generator().manual_seed(2)
    logits = torch.randint(-1, 2, (T, 96), generator=g).float().to(gpu)
    bias = (0.25 * torch.randint(0, 2, (96,), generator=g)).to(gpu)
    Select(logits, 12, softmax).check()
    Select(logits, 12, softmax, bias=torch.zeros(96, device=gpu)).check()
    Select(logits, 7, softmax, 8, 3, 1).check()
    Select(logits, 7, softmax, 8, 3, 2).check()
    Select(logits, 7, softmax, 8, 3, 2, bias=0 * bias).check()
    Select(torch.zeros(T, 96, device=gpu), 5, softmax, 4, 2, 2, bias=bias).check()


@pytest.mark.gpu
@pytest.mark.parametrize("E", [32, 256, 500])
@pytest.mark.parametrize("softmax", [True, False])
def test_close_scores(gpu, softmax, E):
    """A bias that makes every score nearly the same: what float32 leaves open is decided as in 64 bits."""
    logits, _, _ = make(gpu, 1, E, torch.float32, E)
    rows = logits + torch.tensor([[0.0], [2.0 ** -20], [0.0]], device=gpu)
    s = torch.from_numpy(ref.scores(logits.double().cpu().numpy(), softmax)[0])
    bias = (0.7 - s).float().to(gpu)  # sums of 0.7 to within float32's rounding
    Select(rows.contiguous(), 8, softmax, bias=bias).check()
    Select(rows.repeat(100, 1), 8, softmax, bias=bias).check()
    Select(rows.repeat(30, 1), 8, softmax, 4, 2, 2, bias=bias).check()
    Select(rows.repeat(30, 1), 8, softmax, 4, 2, 1, bias=bias).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [9, 150])
def test_all_chosen_side_by_side(gpu, T, dtype):
    """More of the chosen next to each other than a group of lanes keeps sorted for its share."""
    logits, bias, _ = make(gpu, T, 512, dtype, 11)
    rows = torch.arange(T, device=gpu)
    for i in range(14):
        logits[rows, (32 * (rows % 16) + 2 * i) % 512] += 12
    for kw in (dict(), dict(bias=bias), dict(bias=bias, groups=4, top_groups=2, best=2)):
        Select(logits, 16, True, **kw).check()
        Select(logits, 16, False, **kw).check()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(5000, 256, 8), (8200, 60, 6), (300001, 16, 4)])
def test_many_tokens(gpu, T, E, k):
    """Workgroups that go through their tokens in several turns; the choice against a sort, the order against the ids."""
    logits, _, valid = make(gpu, T, E, torch.float32, T)
    x = Select(logits, k, valid=valid)
    x.forward()
    best, at = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = torch.where(valid[:, None], at[:, :k].to(i32), -1)
    assert torch.equal(x.ids, ids)
    w = torch.softmax(best[:, :k].double(), 1) * valid[:, None]
    # The difference of two logits is rounded once, its exponential and the quotient add a few steps.
    assert ((x.w - w).abs() <= (24 + 4 * 12) * ref.U * w).all()
    counts, offsets, order = ref.order(ids.cpu().numpy(), E)
    assert np.array_equal(x.counts.cpu().numpy(), counts) and np.array_equal(x.offsets.cpu().numpy(), offsets)
    places = x.order.cpu().numpy()
    assert np.array_equal(places[:len(order)], order) and (places[len(order):] == -7).all()


@pytest.mark.gpu
def test_close_groups_without_a_bias(gpu):
    """Groups whose sums of two agree to a few steps of float32."""
    g = torch.Generator().manual_seed(5)
    logits = torch.full((64, 40), -8.0)
    a = torch.rand(64, 10, generator=g, dtype=torch.float64) * 2 + 0.5
    # softmax: e^a + e^b the same in every group; the first and the second expert of each.
    logits[:, 0::4] = a.float()
    logits[:, 1::4] = torch.log(16 - torch.exp(a.float().double())).float()
    Select(logits.to(gpu), 6, True, 10, 3, 2).check()
    s = 1 / (1 + torch.exp(-a))
    logits[:, 1::4] = -torch.log(1 / (1.6 - s).clamp(0.05, 0.95) - 1).float()
    Select(logits.to(gpu), 6, False, 10, 3, 2).check()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("T", [4, 100])
def test_excluded_experts(gpu, T, softmax):
    """Logits and biases of -inf, NaN biases, rows with fewer than k experts or none."""
    logits, bias, valid = make(gpu, T, 48, torch.float32, 3)
    inf = float("inf")
    logits[:, 5:9] = -inf
    logits[1] = -inf
    logits[2, 3:] = -inf
    logits[3, 12:] = -inf
    bias[0], bias[10], bias[11] = -inf, float("nan"), inf
    for renorm in (True, False):
        x = Select(logits, 6, softmax, renorm=renorm).check()
        assert (x.ids[1] == -1).all() and not x.w[1].any() and not x.d[1].any() and (x.ids[2, 3:] == -1).all()
        Select(logits, 6, softmax, renorm=renorm, bias=bias, valid=valid).check()
        Select(logits, 6, softmax, 6, 3, 2, renorm=renorm, bias=bias).check()
        Select(logits, 6, softmax, 6, 3, 1, renorm=renorm).check()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_is_not_hidden(gpu, bad, softmax):
    logits, bias, _ = make(gpu, 100, 40, torch.float32, 4)
    logits[7, 3] = bad
    for kw in (dict(), dict(bias=bias), dict(renorm=False), dict(groups=5, top_groups=2, best=2, bias=bias)):
        x = Select(logits, 4, softmax, **kw)
        x.check()
        hidden = bad == bad and not softmax  # a sigmoid of +inf is 1
        assert bool(x.w[7].isnan().all()) != hidden and bool(x.d[7].isnan().all()) != hidden
        assert not x.w[:7].isnan().any() and not x.w[8:].isnan().any() and not x.d[8:].isnan().any()
    valid = torch.ones(100, dtype=torch.uint8, device=gpu)
    valid[7] = 0  # in a padding token's row it does not count
    y = Select(logits, 4, softmax, valid=valid).check()
    assert not y.w.isnan().any() and not y.d[7].any()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
def test_far_logits(gpu, softmax):
    """Scores below float32's range, or next to 1: weights and gradients stay those of the formula."""
    logits, _, _ = make(gpu, 60, 20, torch.float32, 6)
    logits[::3] -= 300
    logits[1::3] += 60
    logits[2::3, 4] += 80
    Select(logits, 4, softmax).check()
    Select(logits, 4, softmax, renorm=False).check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 300])
def test_no_valid_token_no_token_and_no_order(gpu, T):
    logits, bias, _ = make(gpu, T, 40, torch.float32, 1)
    x = Select(logits, 3, valid=torch.zeros(T, dtype=torch.bool, device=gpu)).check()
    assert (x.ids == -1).all() and not x.w.any() and not x.counts.any() and not x.d.any()
    y = Select(logits[:0], 3)
    y.forward()
    y.backward()
    assert not y.counts.any() and not y.offsets.any()
    z, full = Select(logits, 3, bias=bias), Select(logits, 3, bias=bias)
    z.forward(order=False)
    full.forward()
    assert torch.equal(z.ids, full.ids) and torch.equal(z.w, full.w) and (z.counts == -9).all() and (z.order == -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True)])
def test_gradient_in_place(gpu, softmax, renorm, dtype):
    """Into the base's memory, and into the logits'."""
    logits, bias, valid = make(gpu, 500, 200, dtype, 6)
    x = Select(logits, 5, softmax, renorm=renorm, bias=bias, valid=valid, base=True).check()
    want = x.d.clone()
    x.d = x.base
    x.backward()
    assert torch.equal(x.d, want)
    y = Select(logits, 5, softmax, renorm=renorm, bias=bias, valid=valid)
    y.forward()
    y.backward()
    want = y.d
    y.d = y.logits
    y.backward()
    assert torch.equal(y.d, want)


@pytest.mark.gpu
@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True), (False, False)])
def test_gradient_by_differences(gpu, softmax, renorm):
    """The weights' own slope along a direction, of tokens whose choice a step does not change."""
    logits, _, _ = make(gpu, 200, 24, torch.float32, 5)
    x = Select(logits, 3, softmax, renorm=renorm)
    x.forward()
    x.backward()
    way = torch.sign(x.d)
    h = 0.01
    value, same = [], torch.ones(200, dtype=torch.bool, device=gpu)
    for step in (h, -h):
        y = Select(logits + step * way, 3, softmax, renorm=renorm)
        y.forward()
        same &= (y.ids == x.ids).all(1)
        value.append((y.w.double() * x.dw).sum(1))
    assert same.sum() > 100
    slope = (x.d.double() * way).sum(1)
    size = (x.w.double() * x.dw).abs().sum(1)
    # A weight's third derivative along signs is at most 16 times it; weights carry 2^-20 relative.
    far = ((value[0] - value[1]) / (2 * h) - slope).abs() - (16 * h * h * size + 2.0 ** -20 * size / h)
    assert far[same].max() <= 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,E", [(1, 1), (5, 3), (64, 64), (1000, 7), (4096, 512), (4097, 512), (30000, 64), (200001, 2),
                                 (1500000, 300)])
def test_sort(gpu, n, E):
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(-1, E + 1, (n,), generator=g, dtype=i32)  # some outside on both sides
    ids[::17] = min(2, E - 1)
    full = lambda m, v=-9: torch.full((m,), v, dtype=i32, device=gpu)  # noqa: E731
    counts, offsets, order = full(E), full(E + 1), full(n, -7)
    ws = torch.full((moe.moe_sort_workspace_bytes(n, E),), 0xEE, dtype=torch.uint8, device=gpu)
    moe.moe_sort_assignments(ids.to(gpu), E, counts, offsets, order, ws)
    want = ref.order(ids.numpy(), E)
    assert np.array_equal(counts.cpu().numpy(), want[0]) and np.array_equal(offsets.cpu().numpy(), want[1])
    got = order.cpu().numpy()
    assert np.array_equal(got[:len(want[2])], want[2]) and (got[len(want[2]):] == -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 8, 15, 16, 17, 63, 129])
@pytest.mark.parametrize("E", [1, 16, 65, 512])
def test_sort_few(gpu, n, E):
    """Few assignments, those of no expert and equal ones among them; nothing behind what is asked for is written."""
    g = torch.Generator().manual_seed(n * 1000 + E)
    for ids in (torch.randint(-1, E + 1, (n,), generator=g, dtype=i32), torch.full((n,), E - 1, dtype=i32),
                torch.full((n,), 2 ** 31 - 1, dtype=i32)):
        full = lambda m: torch.full((m + 4,), -9, dtype=i32, device=gpu)  # noqa: E731
        counts, offsets, order = full(E), full(E + 1), full(n)
        ws = torch.empty(moe.moe_sort_workspace_bytes(n, E), dtype=torch.uint8, device=gpu)
        moe.moe_sort_assignments(ids.to(gpu), E, counts[:E], offsets[:E + 1], order[:n], ws)
        want = ref.order(ids.numpy(), E)
        for got, exact in zip((counts, offsets, order), want):
            got = got.cpu().numpy()
            assert np.array_equal(got[:len(exact)], exact) and (got[len(exact):] == -9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,k", [(1, 1), (1, 8), (1, 16), (2, 8), (3, 6), (5, 3), (16, 1), (17, 1)])
@pytest.mark.parametrize("groups", [1, 4])
def test_order_of_few(gpu, T, k, groups):
    """The order that comes with a choice for few tokens is that of its ids, rows without an expert among them."""
    logits, bias, _ = make(gpu, T, 64, torch.float32, 31 * T + k)
    x = Select(logits, k, True, groups, 1 if groups == 1 else 2, 1, bias=bias)
    x.forward()
    for _ in range(2):
        want = ref.order(x.ids.cpu().numpy().reshape(-1), 64)
        for got, exact in zip((x.counts, x.offsets, x.order), want):
            assert np.array_equal(got.cpu().numpy()[:len(exact)], exact)
        x.logits[T // 2] = -float("inf")
        x.forward()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [17, 64, 100, 2085, 4096, 4097, 70001])
@pytest.mark.parametrize("runs", [1, 2, 3, 8])
def test_sort_runs(gpu, n, runs):
    """Long runs of one id, some of them no expert's, whose ends lie anywhere in a wave's 64."""
    g = torch.Generator().manual_seed(n + runs)
    cuts = torch.sort(torch.randint(0, n + 1, (runs - 1,), generator=g)).values.tolist()
    values = torch.randint(-1, 9, (runs,), generator=g).tolist()
    ids = torch.cat([torch.full((hi - lo,), v, dtype=i32) for lo, hi, v in zip([0] + cuts, cuts + [n], values)])
    full = lambda m: torch.full((m,), -9, dtype=i32, device=gpu)  # noqa: E731
    counts, offsets, order = full(8), full(9), full(n)
    ws = torch.empty(moe.moe_sort_workspace_bytes(n, 8), dtype=torch.uint8, device=gpu)
    moe.moe_sort_assignments(ids.to(gpu), 8, counts, offsets, order, ws)
    want = ref.order(ids.numpy(), 8)
    assert np.array_equal(counts.cpu().numpy(), want[0]) and np.array_equal(offsets.cpu().numpy(), want[1])
    got = order.cpu().numpy()
    assert np.array_equal(got[:len(want[2])], want[2]) and (got[len(want[2]):] == -9).all()


@pytest.mark.gpu
def test_sort_nothing(gpu):
    counts, offsets = torch.full((6,), 3, dtype=i32, device=gpu), torch.full((7,), 3, dtype=i32, device=gpu)
    empty = torch.empty(0, dtype=i32, device=gpu)
    moe.moe_sort_assignments(empty, 6, counts, offsets, empty, torch.empty(256, dtype=torch.uint8, device=gpu))
    assert not counts.any() and not offsets.any()
    moe.moe_sort_assignments(torch.full((50,), -1, dtype=i32, device=gpu), 6, counts, offsets,
                             torch.empty(50, dtype=i32, device=gpu),
                             torch.empty(moe.moe_sort_workspace_bytes(50, 6), dtype=torch.uint8, device=gpu))
    assert not counts.any() and not offsets.any()


@pytest.mark.gpu
def test_repeat_bits_streams_and_graph(gpu):
    """The same bits from call to call, from two streams at once, and from a graph replayed on new logits."""
    def new(seed):
        la, ba, va = make(gpu, 3000, 256, torch.float32, seed)
        lb, bb, _ = make(gpu, 900, 512, torch.bfloat16, seed + 1)
        return [Select(la, 8, True, valid=va), Select(lb, 4, False, 8, 4, 2, bias=bb, base=True)]

    xs = new(7)
    wants = []
    for x in xs:
        x.forward()
        x.backward()
        wants.append([t.clone() for t in x.outputs()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                x.forward()
                x.backward()
    torch.cuda.synchronize()
    for x, want in zip(xs, wants):
        assert all(torch.equal(t, w) for t, w in zip(x.outputs(), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for x in xs:
            x.forward()
            x.backward()
    for seed in (9, 19, 29):
        ys = new(seed)
        for x, y in zip(xs, ys):
            x.logits.copy_(y.logits)
            x.dw.copy_(y.dw)
            if x.bias is not None:
                x.bias.copy_(y.bias)
            if x.valid is not None:
                x.valid.copy_(y.valid)
            if x.base is not None:
                x.base.copy_(y.base)
            x.order.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(xs, ys):
            y.forward()
            y.backward()
            assert all(torch.equal(a, b) for a, b in zip(x.outputs(), y.outputs()))


@pytest.mark.gpu
def test_unaligned_tensors(gpu):
    """Logits, gradients and ids that begin at odd elements of larger buffers."""
    for dtype in (torch.float32, torch.bfloat16):
        logits, bias, valid = make(gpu, 90, 129, dtype, 8)
        x = Select(logits, 5, False, 3, 2, 2, bias=bias, valid=valid, base=True)
        for name in ("logits", "w", "ids", "dw", "d", "base", "order", "counts", "offsets"):
            t = getattr(x, name)
            odd = torch.empty(t.numel() + 1, dtype=t.dtype, device=gpu)[1:].view(t.shape)
            odd.copy_(t)
            setattr(x, name, odd)
        x.check()


@pytest.mark.gpu
def test_same_choice_as_the_layers_router(gpu):
    """From the router's own logits: its ids, weights and metadata."""
    import moe_inputs as mi
    from bit_quantized_moe_router_amd.layer import MoELayer, to_dev

    case = mi.make_case("tiny")
    lay = MoELayer(case["w"], case["k"], device=gpu, max_tokens=64)
    x = to_dev(case["x"], gpu)
    r = lay.route(x)
    logits = (x.view(torch.bfloat16).double() @ lay.router_w.double().t()).float().contiguous()
    s = Select(logits, case["k"]).check()
    assert torch.equal(s.ids, r["topk_ids"]) and torch.equal(s.counts, r["expert_counts"])
    assert torch.equal(s.offsets, r["expert_offsets"]) and torch.equal(s.order, r["sorted_assign"])
    assert (s.w - r["topk_weights"]).abs().max() <= 2.0 ** -20


@pytest.mark.gpu
@pytest.mark.parametrize("among", [1, 2])
@pytest.mark.parametrize("k", [1, 2, 3, 5, 8, 16])
def test_three_close_around_the_last_place(gpu, k, among):
    """Three experts a step of float32 apart, of which `among` are to be chosen, in any order, with all others far off."""
    g = torch.Generator().manual_seed(100 * k + among)
    T, E, above = 400, 64, max(0, k - among)
    close = torch.tensor([1.0, 1.0 + 2.0 ** -23, 1.0 + 2.0 ** -22])
    rows = torch.empty(T, E)
    for t in range(T):
        places = torch.randperm(E, generator=g)
        rows[t, places[:above]] = 2 + torch.rand(above, generator=g)
        rows[t, places[above:above + 3]] = close[torch.randperm(3, generator=g)]
        rows[t, places[above + 3:]] = -torch.rand(E - above - 3, generator=g)
    rows = rows.to(gpu)
    for softmax in (True, False):
        Select(rows, k, softmax).check()
        Select(rows[:7].contiguous(), k, softmax).check()
        # Of all groups but one, the same within them.
        Select(rows, k, softmax, 4, 3, 1).check()
    # Scores of a sigmoid that differ in their last bits, with a bias that is the same for the three.
    near = rows.clone()
    for v, l in zip(close.tolist(), (16.0, 16.125, 16.25)):
        near[rows == v] = l
    for dtype in (torch.float32, torch.bfloat16):
        # The bias lifts the experts above the three by one.
        l = near.to(dtype)
        for t in range(0, 40):
            bias = 0.25 + (rows[t] >= 2).float()
            Select(l[t:t + 1].contiguous(), k, False, bias=bias).check()
            Select(l[t:t + 1].contiguous(), k, True, bias=bias).check()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("dtype,lowest", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                          (torch.float32, torch.float32)])
@pytest.mark.parametrize("T", [6, 130])
def test_masks_of_the_lowest_value(gpu, T, dtype, lowest, softmax):
    """A logit of the type's lowest value is an expert like any other: chosen where there are no k better ones."""
    logits, bias, _ = make(gpu, T, 48, torch.bfloat16, 12)
    logits = logits.to(dtype)
    low, inf = torch.finfo(lowest).min, float("inf")
    logits[0] = low
    logits[1::2, 4:] = low
    logits[2::4, :46] = low
    logits[3::4, 2] = -inf
    logits[3::4, 20:] = -inf
    some = (logits.float() > low).sum(1, keepdim=True)
    for kw in (dict(), dict(renorm=False), dict(bias=bias), dict(groups=6, top_groups=3), dict(groups=6, top_groups=3, best=2),
               dict(groups=6, top_groups=3, best=2, bias=bias)):
        x = Select(logits, 8, softmax, **kw).check()
        assert (x.ids >= 0).all()
        if "bias" in kw or "groups" in kw:
            continue
        # Their scores are zeros, but where there are no others: those are the same for all.
        place = torch.arange(8, device=gpu)
        assert not x.w[(place >= some) & (some > 0)].any()
        if not kw:
            assert ((x.w[0] - 1 / 8).abs() <= 2.0 ** -24).all()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("lo,hi", [(-3.0, -2.9), (-5.0, -4.8), (-100.0, -99.0), (2.9, 3.1), (1.0, 1.2), (0.5, 0.51), (99.0, 100.0),
                                   (1000.0, 1001.0), (-1e6, 1 - 1e6), (1e9, 1.1e9), (-3e38, 3e38), (1e-30, 2e-30)])
def test_biases_far_from_zero(gpu, lo, hi, softmax):
    """Scores too small to change their sum with the bias, where every expert is to be chosen, or some of them."""
    g = torch.Generator().manual_seed(3)
    for T in (5, 150):
        for E, k in ((16, 16), (64, 16), (16, 5)):
            logits = -17 - 8 * torch.rand(T, E, generator=g)
            logits[torch.arange(T), torch.randint(0, E, (T,), generator=g)] = 1.0
            bias = (torch.rand(E, generator=g).double() * (hi - lo) + lo).float()
            bias[E // 2] = lo
            bias, logits = bias.to(gpu), logits.to(gpu)
            for kw in (dict(), dict(groups=4, top_groups=4)) + ((dict(groups=4, top_groups=2, best=2),) if k != 16 or E == 64 else ()):
                for dtype in (torch.float32, torch.bfloat16):
                    x = Select(logits.to(dtype), k, softmax, bias=bias, **kw).check()
                    assert (x.ids >= 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("value", [0.0, 0.5, -3.0, 1.0, 1e10])
def test_one_bias_for_all(gpu, value, softmax):
    """The choice is that of the float64 sums: scores that do not differ in them are equal, whatever their logits."""
    logits, _, _ = make(gpu, 60, 20, torch.float32, 6)
    logits[::3] -= 300
    logits[1::3] += 60
    logits[2::3, 4] += 80
    for T in (60, 3):
        for dtype in (torch.float32, torch.bfloat16):
            l = logits[:T].to(dtype)
            bias = torch.full((20,), value, device=gpu)
            Select(l, 4, softmax, bias=bias).check()
            Select(l, 4, softmax, 5, 2, 2, bias=bias).check()
    # Groups that have one expert left: their sum has the bias once.
    few = torch.randn(60, 8, generator=torch.Generator().manual_seed(1)).to(gpu)
    few[:, 1] = -float("inf")
    few[::2, 4] = -float("inf")
    for T in (60, 3):
        Select(few[:T].contiguous(), 2, softmax, 4, 2, 2, bias=torch.full((8,), value, device=gpu)).check()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("scale", [1e-39, -3e-40, 1e30])
def test_gradient_of_extreme_scales(gpu, scale, softmax):
    """A scale whose reciprocal float32 does not hold."""
    logits, _, _ = make(gpu, 100, 24, torch.float32, 15)
    x = Select(logits, 5, softmax, scale=scale)
    x.forward()
    x.dw /= abs(x.desc.scale) * 64  # gradients near 1
    x.backward()
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    # For the weights as they were written: subnormal ones hold few bits.
    want, size = ref.select_gradient(n(logits), x.ids.cpu().numpy(), n(x.w), n(x.dw), softmax, True, x.desc.scale)
    # Five products and their sum, a quotient, a difference and a product; 1 - s by an exponential of an argument below 8.
    assert (np.abs(n(x.d) - want) <= 64 * ref.U * size + 1e-37).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,n,top,k", GROUPS)
def test_groups_of_sigmoid_sums(gpu, T, E, n, top, k, dtype):
    """Ranked by sums of two sigmoid scores without a bias; logits of one sign, as sums for x and -x are all 1."""
    logits, _, valid = make(gpu, T, E, torch.float32, T + E)
    for sign in (1, -1):
        l = (sign * logits.abs()).to(dtype)
        Select(l, k, False, n, top, 2, valid=valid).check()
        Select(l, k, False, n, top, 2, renorm=False, scale=2.5).check()


@pytest.mark.gpu
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("T", [40, 700])
def test_equal_sums_beside_close_ones(gpu, T, softmax):
    """Equal logits with equal biases, two of them or many around the last place, among others as close as float32 tells."""
    g = torch.Generator().manual_seed(T)
    for dtype in (torch.float32, torch.bfloat16):
        for E, k in ((32, 6), (96, 16), (256, 8)):
            few = torch.randint(0, 24, (T, E), generator=g).float() * 0.25
            few[T // 2:] += 13  # a sigmoid's last bits
            few[::3] += (torch.rand(len(few[::3]), E, generator=g) < 0.1) * 2.0 ** -20
            for bias in (torch.zeros(E), torch.full((E,), 0.5), 0.25 * torch.randint(0, 2, (E,), generator=g).float()):
                l, b = few.to(dtype).to(gpu), bias.to(gpu)
                Select(l, k, softmax, bias=b).check()
                Select(l, k, softmax, 4, 2, 1, bias=b).check()
