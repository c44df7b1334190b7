"""Tokens sorted by expert and back on the GPU: the split against a stable sort, the moves bit for bit, the sums
against 64 bits."""
import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
from sequence_reference import HALF, TINY, U, f64

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def randn(rng, *shape, t=torch.float32, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(t).cuda()


def wider(x, left=8, right=8):
    """x as a slice of a tensor with more columns, which hold NaN."""
    w = torch.full(x.shape[:-1] + (left + x.shape[-1] + right,), float("nan"), dtype=x.dtype, device=x.device)
    w[..., left:left + x.shape[-1]] = x
    return w[..., left:left + x.shape[-1]]


def within(got, want, error, what):
    """`got` within the error of `want` before the rounding to its type."""
    t = got.dtype
    bad = ~(np.abs(f64(got) - want) <= error + HALF[t] * (np.abs(want) + error) + TINY[t])
    assert not bad.any(), "%s: %d of %d values outside" % (what, bad.sum(), bad.size)


def split_reference(experts, e):
    """(offsets, places, source) by a stable sort."""
    flat = experts.reshape(-1).astype(np.int64)
    bucket = np.where((flat >= 0) & (flat < e), flat, e)
    order = np.argsort(bucket, kind="stable")
    offsets = np.searchsorted(bucket[order], np.arange(e + 1))
    total = int(offsets[e])
    source = np.full(flat.size, -1)
    source[:total] = order[:total]
    places = np.full(flat.size, -1)
    places[order[:total]] = np.arange(total)
    return offsets, places.reshape(experts.shape), source


def choices(rng, kind, n, k, e):
    if kind == "uniform":
        c = rng.integers(-1, e + 1, (n, k))
    elif kind == "one":
        c = np.full((n, k), e // 2)
    elif kind == "none":
        c = np.where(rng.integers(0, 2, (n, k)) == 0, -2 ** 31, 2 ** 31 - 1)
    elif kind == "last":
        c = np.full((n, k), e - 1)
    else:  # falling frequencies
        c = np.minimum((e * rng.uniform(0, 1, (n, k)) ** 4).astype(np.int64), e - 1)
    return c.astype(np.int32)


def split_check(plan, experts, e):
    for name, got, want in zip(plan._fields, plan, split_reference(experts, e)):
        assert got.dtype == torch.int32 and got.shape == want.shape, name
        assert np.array_equal(got.cpu().numpy(), want), name


# 4096 choices to a chunk; more than 64 chunks take a launch of their own for the prefixes
@pytest.mark.parametrize("kind", ["uniform", "one", "none", "last", "skewed"])
@pytest.mark.parametrize("n,k,e", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (13, 5, 3), (64, 1, 64), (65, 1, 65), (512, 8, 256), (4097, 1, 7),
                                   (2049, 2, 1024), (1000, 20, 1000), (9000, 8, 100), (70001, 4, 33), (270001, 1, 2)])
def test_split(kind, n, k, e):
    rng = np.random.default_rng(n + k + e)
    c = choices(rng, kind, n, k, e)
    plan = dw.expert_split(torch.from_numpy(c).cuda(), e)
    split_check(plan, c, e)


def setup(rng, n, k, e, d, t, weight_t=torch.float32):
    c = choices(rng, "uniform", n, k, e)
    plan = dw.expert_split(torch.from_numpy(c).cuda(), e)
    y = randn(rng, n * k, d, t=t)
    y[int(plan.offsets[-1]):] = float("nan")  # rows of no expert hold anything
    return plan, randn(rng, n, d, t=t), y, randn(rng, n, k, t=weight_t), randn(rng, n, d, t=t)


SIZES = [(1, 1, 1, 1), (3, 2, 4, 8), (70, 8, 16, 64), (33, 5, 7, 515), (20, 3, 5, 590), (9, 9, 12, 2056), (40, 2, 8, 1002), (5, 20, 30, 136),
         (2, 256, 300, 24), (600, 4, 32, 72)]


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("n,k,e,d", SIZES)
def test_dispatch(t, n, k, e, d):
    rng = np.random.default_rng(n + k + d)
    t = T[t]
    plan, x, _, _, _ = setup(rng, n, k, e, d, t)
    total = int(plan.offsets[-1])
    token = (plan.source[:total] // k).long()
    for src in (x, wider(x)):
        rows = dw.expert_dispatch(src, plan)
        assert rows.shape == (n * k, d) and torch.equal(rows[:total], x[token]) and (rows[total:] == 0).all()
    wide = torch.full((n * k + 3, d + 6), 5.0, dtype=t, device="cuda")
    out = wide[:, 2:2 + d]
    assert dw.expert_dispatch(x, plan, out=out) is out
    assert torch.equal(out[:total], x[token])
    wide[:total, 2:2 + d] = 5.0
    assert (wide == 5.0).all()  # rows of no expert and columns beside are left as they were


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("n,k,e,d", SIZES)
def test_combine_and_gradients(t, n, k, e, d):
    rng = np.random.default_rng(n + k + d + 1)
    t = T[t]
    for weight_t, strided in ((torch.float32, True), (t, False), (None, False)):
        plan, x, y, w, dout = setup(rng, n, k, e, d, t, weight_t or torch.float32)
        if strided:
            y, dout = wider(y), wider(dout)
        weights = None if weight_t is None else w
        places = plan.places.cpu().numpy()
        there = (places >= 0)[..., None]
        w64 = np.where(there, 1.0 if weight_t is None else f64(w)[..., None], 0.0)
        rows = np.where(there, np.nan_to_num(f64(y))[places.clip(min=0)], 0.0)
        terms = w64 * rows
        # k fused multiply-adds, one rounding each
        out = dw.expert_combine(y, plan, weights)
        within(out, terms.sum(1), (k + 1) * U * np.abs(terms).sum(1), "combine")
        given = torch.full((n, d + 5), 3.0, dtype=t, device="cuda")
        dw.expert_combine(y, plan, weights, out=given[:, :d])
        assert torch.equal(given[:, :d], out) and (given[:, d:] == 3.0).all()

        g = dw.expert_combine_grad(dout, y, plan, weights)
        total = int(plan.offsets[-1])
        source = plan.source[:total].long()
        product = dout[source // k].float() * (1.0 if weight_t is None else w.float().reshape(-1)[source][:, None])
        assert g.dy.shape == y.shape and torch.equal(g.dy[:total], product.to(t)) and (g.dy[total:] == 0).all()
        if weight_t is None:
            assert g.dweights is None
        else:
            # a thread's share of the channels one after another, 6 sums over lanes, 3 over wavefronts
            sums = np.where(there, rows * f64(dout)[:, None], 0.0)
            assert g.dweights.dtype == torch.float32
            within(g.dweights, sums.sum(-1), (d / 256 + 8 + 6 + 3 + 2) * U * np.abs(sums).sum(-1), "dweights")
            assert (g.dweights[plan.places < 0] == 0).all()
        dy = torch.full((n * k, d), 4.0, dtype=t, device="cuda")
        g2 = dw.expert_combine_grad(dout, y, plan, weights, dy=dy)
        assert g2.dy is dy and torch.equal(dy[:total], g.dy[:total]) and (dy[total:] == 4.0).all()

        ones = np.where(there, rows, 0.0)
        dx = dw.expert_dispatch_grad(y, plan)
        within(dx, ones.sum(1), (k + 1) * U * np.abs(ones).sum(1), "dispatch gradient")
        assert dw.expert_dispatch_grad(y, plan, dx=x) is x and torch.equal(x, dx)
        for _ in range(2):
            assert torch.equal(dw.expert_combine(y, plan, weights), out)


def test_gradients_are_adjoints():
    """Both moves are linear: the product of an output's change with a gradient is the product of the input's change with
    the gradient passed back, up to the roundings of each."""
    rng = np.random.default_rng(5)
    plan, x, y, w, dout = setup(rng, 200, 6, 16, 100, torch.float32)
    y = torch.nan_to_num(y)
    drows = randn(rng, 1200, 100)
    total = int(plan.offsets[-1])
    rows, dx = dw.expert_dispatch(x, plan), dw.expert_dispatch_grad(drows, plan)
    lhs, rhs = f64(rows) * f64(drows), f64(x) * f64(dx)
    assert abs(lhs[:total].sum() - rhs.sum()) <= 8 * U * (np.abs(lhs).sum() + np.abs(rhs).sum())
    out, g = dw.expert_combine(y, plan, w), dw.expert_combine_grad(dout, y, plan, w)
    a, b, c = f64(out) * f64(dout), f64(y) * f64(g.dy), f64(w) * f64(g.dweights)
    terms = np.abs(f64(w))[..., None] * np.abs(f64(y))[plan.places.cpu().numpy().clip(min=0)] * np.abs(f64(dout))[:, None]
    assert abs(a.sum() - b.sum()) <= 8 * U * terms.sum()
    assert abs(a.sum() - c.sum()) <= 24 * U * terms.sum()


def test_plans_of_other_origin():
    """Places outside the rows are skipped, in a plan with room between the experts too; a place met twice holds either's."""
    rng = np.random.default_rng(6)
    x = randn(rng, 4, 40)
    places = torch.tensor([[0, 9], [3, -1], [3, 100], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    plan = dw.ExpertPlan(torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda"), places, torch.zeros(8, dtype=torch.int32, device="cuda"))
    out = torch.full((10, 40), 2.0, device="cuda")
    dw.expert_dispatch(x, plan, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[9], x[0]) and (torch.equal(out[3], x[1]) or torch.equal(out[3], x[2]))
    assert (out[[1, 2, 4, 5, 6, 7, 8]] == 2.0).all()
    y = dw.expert_combine(out, plan)
    assert torch.equal(y[0], out[0] + out[9]) and torch.equal(y[1], out[3]) and torch.equal(y[2], out[3]) and (y[3] == 0).all()
    # a number of rows outside the array clears nothing outside it
    for end in (-5, 12, 2 ** 31 - 1):
        plan = plan._replace(offsets=torch.tensor([0, end], dtype=torch.int32, device="cuda"), places=places[:, :1].contiguous())
        rows = dw.expert_dispatch(x, plan)
        assert rows.shape == (4, 40) and torch.equal(rows[0], x[0] if end >= 0 else rows[0])


def test_no_tokens():
    plan = dw.expert_split(torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 4)
    assert (plan.offsets == 0).all()
    x = torch.zeros(0, 16, device="cuda")
    assert dw.expert_dispatch(x, plan).shape == (0, 16) and dw.expert_combine(x, plan, torch.zeros(0, 3, device="cuda")).shape == (0, 16)
    given = torch.full((5, 16), 2.0, device="cuda")
    assert (dw.expert_dispatch(x, plan, out=given) == 2.0).all()


def test_values_that_are_not_finite_stay_in_their_tokens():
    rng = np.random.default_rng(7)
    plan, x, y, w, dout = setup(rng, 50, 4, 8, 72, torch.float32)
    clean = dw.expert_combine(y, plan, w)
    place = int(plan.places[plan.places >= 0][5])
    token = int(plan.source[place]) // 4
    y[place, 9] = float("nan")
    out = dw.expert_combine(y, plan, w)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[token, 9] = True
    assert out[hit].isnan().all() and torch.equal(out[~hit], clean[~hit])


def test_offsets_past_32_bits():
    rng = np.random.default_rng(8)
    rows, d = 540001, 4096
    big = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")  # 2.2e9 elements
    x = randn(rng, 2, d, t=torch.bfloat16)
    places = torch.tensor([[rows - 1, 5], [rows - 3, rows - 2]], dtype=torch.int32, device="cuda")
    plan = dw.ExpertPlan(torch.tensor([0, rows], dtype=torch.int32, device="cuda"), places, places.view(-1))
    dw.expert_dispatch(x, plan, out=big)
    assert torch.equal(big[rows - 1], x[0]) and torch.equal(big[5], x[0]) and torch.equal(big[rows - 2], x[1])
    assert torch.equal(dw.expert_combine(big, plan), 2 * x)
    w = torch.ones(2, 2, device="cuda")
    g = dw.expert_combine_grad(x, big, plan, w, dy=torch.empty_like(big))
    assert torch.equal(g.dy[rows - 3], x[1])
    sq = (f64(x) ** 2).sum(-1)
    within(g.dweights, np.stack([sq, sq], 1), (d / 256 + 19) * U * np.stack([sq, sq], 1), "dweights")


def layer(x, experts, weights, e, dout):
    """Forwards and backwards with an expert's product of its own (a factor per expert, exact in the type)."""
    plan = dw.expert_split(experts, e)
    rows = dw.expert_dispatch(x, plan)
    y = rows * 2
    out = dw.expert_combine(y, plan, weights)
    g = dw.expert_combine_grad(dout, y, plan, weights)
    return [plan.offsets, plan.places, rows, out, g.dy, g.dweights, dw.expert_dispatch_grad(g.dy * 2, plan)]


def test_graphs_and_streams():
    rng = np.random.default_rng(9)
    sets = []
    for n, k, e, d in ((300, 4, 16, 64), (3000, 8, 64, 40)):
        c = torch.from_numpy(choices(rng, "uniform", n, k, e)).cuda()
        sets.append((randn(rng, n, d, t=torch.bfloat16), c, randn(rng, n, k), e, randn(rng, n, d, t=torch.bfloat16)))
    eager = [layer(*s) for s in sets]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for s in sets:
            layer(*s)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(layer(*s))
            graphs.append(g)
    torch.cuda.synchronize()
    for turn in range(4):
        for o in outs:
            for q in o:
                q.fill_(7)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        if turn % 2:
            layer(*sets[1])
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, eager):
            assert all(torch.equal(p, q) for p, q in zip(o, w))
    plan = dw.expert_split(sets[1][1], 64, stream=other.cuda_stream)
    rows = dw.expert_dispatch(sets[1][0], plan, stream=other)
    other.synchronize()
    assert torch.equal(plan.places, eager[1][1]) and torch.equal(rows, eager[1][2])


def test_gradients_against_autograd_of_the_formulas():
    """Router weights, experts and rows in 64 bits on the host: k + d products and sums relative to the largest."""
    rng = np.random.default_rng(10)
    n, k, e, d = 60, 3, 8, 40
    c = choices(rng, "uniform", n, k, e)
    x, w, dout = randn(rng, n, d), randn(rng, n, k), randn(rng, n, d)
    got = layer(x, torch.from_numpy(c).cuda(), w, e, dout)
    lx, lw = (q.double().cpu().requires_grad_() for q in (x, w))
    there = torch.from_numpy((c >= 0) & (c < e)).double()
    out = (lx[:, None] * 2 * (lw * there)[..., None]).sum(1)
    gx, gw = torch.autograd.grad(out, (lx, lw), dout.double().cpu())
    for g, want in ((got[3], out.detach()), (got[5], gw), (got[6], gx)):
        assert (g.double().cpu() - want).abs().max() <= 2 ** -24 * (k + d) * 4 * max(1.0, float(want.abs().max()))


def test_refusals():
    rng = np.random.default_rng(11)
    plan, x, y, w, dout = setup(rng, 6, 2, 4, 16, torch.float32)
    c = plan.places.clone()
    for bad in (lambda: dw.expert_split(c.long(), 4), lambda: dw.expert_split(c.view(-1), 4), lambda: dw.expert_split(c, 0),
                lambda: dw.expert_split(c, 1025), lambda: dw.expert_split(c.t(), 4), lambda: dw.expert_split(c.cpu(), 4),
                lambda: dw.expert_dispatch(x[:5], plan), lambda: dw.expert_dispatch(x.double(), plan), lambda: dw.expert_dispatch(x.cpu(), plan),
                lambda: dw.expert_dispatch(x, plan, out=y.half()), lambda: dw.expert_dispatch(x, plan, out=y[:, :8]), lambda: dw.expert_dispatch(x.t(), plan),
                lambda: dw.expert_dispatch(x, plan._replace(places=c.long())), lambda: dw.expert_dispatch(x, plan._replace(offsets=c)),
                lambda: dw.expert_combine(y, plan, w.double()), lambda: dw.expert_combine(y, plan, w[:, :1]), lambda: dw.expert_combine(y, plan, w.cpu()),
                lambda: dw.expert_combine(y, plan, w, out=x[:5]), lambda: dw.expert_combine(y, plan, w, out=y[:6]),
                lambda: dw.expert_combine_grad(dout, y[:, :8], plan, w), lambda: dw.expert_combine_grad(dout[:5], y, plan, w),
                lambda: dw.expert_combine_grad(dout, y, plan, w, dy=y), lambda: dw.expert_combine_grad(dout, y.half(), plan, w),
                lambda: dw.expert_dispatch_grad(y, plan, dx=x[:5]), lambda: dw.expert_combine(y.clone().requires_grad_(), plan, w)):
        with pytest.raises((TypeError, ValueError, dw.ScanError)):
            bad()
    assert torch.isfinite(dw.expert_combine(y, plan, w)).all()
