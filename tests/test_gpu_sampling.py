"""Sampling on the GPU against its definition in 64 bits (sampling_reference.py)."""
import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import sampling_reference as sr

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = float("inf")


def make(rng, rows, n, t, std=2.0, peaks=8):
    z = rng.standard_normal((rows, n)) * std
    for r in range(rows):
        z[r, rng.integers(0, n, peaks)] += 6.0
    return torch.from_numpy(z).to(t).cuda()


def uniforms(rng, rows):
    return torch.from_numpy(rng.random(rows).astype(np.float32)).cuda()


def check(logits, u, got, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    z, u, got = logits.double().cpu().numpy(), u.double().cpu().numpy(), got.cpu().numpy()
    rows = z.shape[0]
    wide = lambda q: np.broadcast_to(q.double().cpu().numpy() if torch.is_tensor(q) else q, (rows,))  # noqa: E731
    temperature, top_k, top_p, min_p = (wide(q) for q in (temperature, top_k, top_p, min_p))
    for r in range(rows):
        s = (float(temperature[r]), int(top_k[r]), float(top_p[r]), float(min_p[r]))
        assert sr.accepted(z[r], u[r], int(got[r]), *s), "row %d: %d, not %d, for u %r and settings %r" % (
            r, got[r], sr.token(z[r], u[r], *s)[0], u[r], s)


SETTINGS = [dict(), dict(temperature=0.7), dict(temperature=1.5, top_k=5), dict(top_k=1), dict(top_k=50, top_p=0.9), dict(top_p=0.95),
            dict(temperature=0.6, top_p=0.3), dict(min_p=0.05), dict(temperature=0.9, top_k=200, top_p=0.8, min_p=0.02), dict(temperature=0.0),
            dict(top_k=2000), dict(top_k=1500, top_p=0.5)]


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("rows,n", [(3, 1), (4, 2), (5, 3), (9, 17), (20, 255), (17, 1000), (6, 4097), (40, 8193), (3, 50001), (2, 131072), (2, 200003)])
def test_settings(t, rows, n):
    rng = np.random.default_rng(rows + n)
    logits, u = make(rng, rows, n, T[t]), uniforms(rng, rows)
    for s in SETTINGS:
        got = dw.sample_tokens(logits, u, **s)
        assert got.shape == (rows,) and got.dtype == torch.int32
        check(logits, u, got, **s)


@pytest.mark.parametrize("t", list(T))
def test_settings_of_rows_and_strides(t):
    """Settings per row; rows that start anywhere (odd strides, slices that do not start on 16 bytes)."""
    rng = np.random.default_rng(1)
    for n, left, right in ((1001, 0, 0), (1000, 3, 4), (4096, 1, 6), (777, 5, 0)):
        rows = 48
        whole = torch.full((rows, left + n + right), 99.0, dtype=T[t], device="cuda")  # beside the rows: larger than any logit
        logits = whole[:, left:left + n]
        logits.copy_(make(rng, rows, n, T[t]))
        pick = lambda *of: torch.tensor(of, device="cuda")[torch.from_numpy(rng.integers(0, len(of), rows)).cuda()]  # noqa: E731
        s = dict(temperature=pick(0.0, 0.5, 1.0, 2.0), top_k=pick(-1, 0, 1, 7, 300, 5000).int(), top_p=pick(0.0, 0.5, 0.9, 1.0),
                 min_p=pick(0.0, 0.1, 1.0))
        u = uniforms(rng, rows)
        got = dw.sample_tokens(logits, u, **s)
        check(logits, u, got, **s)
        out = torch.full((rows,), -7, dtype=torch.int64, device="cuda")
        assert dw.sample_tokens(logits, u, out=out, **s) is out and torch.equal(out, got.long())


def test_every_share_of_equal_weights():
    """Logits that are all equal: the token is the index at the random number's share, exactly, with every setting that
    cuts (ties go to the lowest index), also where more tokens tie than the kernel lists."""
    for n in (1, 8, 1000, 4097, 6000, 100000):
        rows = 200
        u = torch.arange(rows, device="cuda", dtype=torch.float32) / rows
        for t in T.values():
            for value in (0.0, -3.0, 7.5):
                logits = torch.full((rows, n), value, dtype=t, device="cuda")
                for s, kept in ((dict(), n), (dict(top_k=max(1, n // 3)), max(1, n // 3)), (dict(top_p=0.5), (n + 1) // 2), (dict(min_p=1.0), n),
                                (dict(top_k=max(1, n // 2), top_p=0.25), max(1, (n // 2 + 3) // 4)), (dict(top_p=0.0), 1)):
                    got = dw.sample_tokens(logits, u, **s).cpu().numpy()
                    want = np.floor(u.double().cpu().numpy() * kept)
                    assert np.array_equal(got, want), (n, t, value, s)


def test_ties_at_the_border():
    """Few distinct logits: the border runs through hundreds of equal ones."""
    rng = np.random.default_rng(2)
    rows, n = 64, 20011
    u = uniforms(rng, rows)
    for t in T.values():
        logits = torch.from_numpy(rng.integers(-6, 3, (rows, n)) * 0.5).to(t).cuda()
        for s in (dict(top_k=3000), dict(top_p=0.6), dict(top_k=10000, top_p=0.7, temperature=2.0), dict(top_k=37), dict(top_p=0.01)):
            check(logits, u, dw.sample_tokens(logits, u, **s), **s)


def test_both_zeros_are_one_logit():
    rows, n = 100, 64
    u = torch.arange(rows, device="cuda", dtype=torch.float32) / rows
    logits = torch.zeros(rows, n, device="cuda")
    logits[:, ::2] = -0.0
    for s, kept in ((dict(top_k=10), 10), (dict(top_p=0.5), 32)):
        assert np.array_equal(dw.sample_tokens(logits, u, **s).cpu().numpy(), np.floor(u.double().cpu().numpy() * kept))
    assert (dw.sample_tokens(logits, u, temperature=0.0) == 0).all()


@pytest.mark.parametrize("t", list(T))
def test_masks_infinities_and_nan(t):
    rng = np.random.default_rng(3)
    t, n = T[t], 3000
    base = make(rng, 1, n, t)[0]
    low = torch.finfo(t).min
    rows = []

    def row(f):
        z = base.clone()
        f(z)
        rows.append(z)

    def only(z, at, rest):
        keep = z[at].clone()
        z.fill_(rest)
        z[at] = keep
    row(lambda z: z.fill_(-INF))
    row(lambda z: z.fill_(float("nan")))
    row(lambda z: only(z, [5], -INF))
    row(lambda z: only(z, [5, 2999], float("nan")))
    row(lambda z: only(z, list(range(100, 140)), low))
    row(lambda z: z.fill_(low))
    row(lambda z: only(z, [7, 8], low) or z[:5].fill_(-INF))
    row(lambda z: z[[3, 900, 901]].fill_(INF) if False else z.index_fill_(0, torch.tensor([3, 900, 901], device="cuda"), INF))
    row(lambda z: z.index_fill_(0, torch.tensor([0, 17], device="cuda"), float("nan")))
    row(lambda z: z[1:].fill_(-INF))
    row(lambda z: z[:-1].fill_(-INF))
    row(lambda z: z.fill_(torch.finfo(t).max))
    row(lambda z: (z[::2].fill_(-INF), z[1::4].fill_(low)))
    logits = torch.stack(rows)
    m = logits.shape[0]
    for value in (0.0, 0.3, 0.77, 1.0 - 2.0 ** -24):
        u = torch.full((m,), value, device="cuda")
        for s in SETTINGS + [dict(top_k=2), dict(top_p=1e-6), dict(temperature=1e-30), dict(temperature=1e30), dict(temperature=INF),
                             dict(temperature=INF, top_k=3)]:
            got = dw.sample_tokens(logits, u, **s)
            check(logits, u, got, **s)
            assert (got[:2] == -1).all() and int(got[2]) == 5 and int(got[9]) == 0 and int(got[10]) == n - 1


def test_random_numbers_at_and_outside_their_range():
    rng = np.random.default_rng(4)
    values = [0.0, -1.0, float("nan"), 2.0 ** -30, 1.0 - 2.0 ** -24, 1.0, 5.0, INF, -INF]
    logits = make(rng, 1, 5001, torch.float32).expand(len(values), -1).contiguous()
    logits[:, 0], logits[:, -1] = 3.0, 3.0
    u = torch.tensor(values, device="cuda")
    for s in (dict(), dict(top_k=4), dict(top_p=0.9), dict(min_p=0.01)):
        got = dw.sample_tokens(logits, u, **s)
        z = logits[0].double().cpu().numpy()
        first, last = sr.token(z, 0.0, 1.0, *(s.get(q, v) for q, v in (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))))[0], None
        last = sr.token(z, 1.0, 1.0, *(s.get(q, v) for q, v in (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))))[0]
        got = got.tolist()
        assert [got[i] for i in (0, 1, 2, 8)] == [first] * 4 and [got[i] for i in (5, 6, 7)] == [last] * 3
        check(logits, u, dw.sample_tokens(logits, u, **s), **s)


def test_settings_at_and_outside_their_range():
    rng = np.random.default_rng(5)
    rows, n = 30, 2000
    logits, u = make(rng, rows, n, torch.float32), uniforms(rng, rows)
    full = dw.sample_tokens(logits, u)
    for s in (dict(top_k=n), dict(top_k=n + 5), dict(top_k=-3), dict(top_p=1.0), dict(top_p=3.0), dict(top_p=float("nan")), dict(min_p=-1.0),
              dict(min_p=0.0), dict(min_p=float("nan")), dict(top_k=2 ** 40)):
        assert torch.equal(dw.sample_tokens(logits, u, **s), full), s
    greedy = logits.argmax(1).int()
    for s in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_k=1), dict(top_p=0.0), dict(top_p=-2.0),
              dict(min_p=1.0), dict(min_p=7.0), dict(temperature=1e-38)):
        assert torch.equal(dw.sample_tokens(logits, u, **s), greedy), s


def test_shares_of_the_whole_distribution():
    """Random numbers in the middle of every token's share give that token, of kept shares too."""
    rng = np.random.default_rng(6)
    n = 300
    z = make(rng, 1, n, torch.float32, std=1.0)[0]
    for s, keep in ((dict(), None), (dict(top_k=20), 20)):
        w = np.exp(z.double().cpu().numpy())
        if keep:
            w[np.argsort(-w, kind="stable")[keep:]] = 0
        run = np.cumsum(w) / w.sum()
        at = np.nonzero(w)[0]
        u = torch.from_numpy((run[at] - 0.5 * w[at] / w.sum()).astype(np.float32)).cuda()
        got = dw.sample_tokens(z.expand(at.size, n).contiguous(), u, **s)
        assert np.array_equal(got.cpu().numpy(), at)


def test_largest_vocabulary():
    rng = np.random.default_rng(7)
    n = 1 << 19
    for t in T.values():
        logits, u = make(rng, 3, n, t), uniforms(rng, 3)
        for s in (dict(), dict(top_p=0.9), dict(top_k=70), dict(temperature=3.0, top_k=100000, top_p=0.5, min_p=1e-5)):
            check(logits, u, dw.sample_tokens(logits, u, **s), **s)


def test_many_rows_and_offsets_past_32_bits():
    rng = np.random.default_rng(8)
    rows, n = 70001, 33000  # 2.3e9 elements
    logits = torch.full((rows, n), -50.0, dtype=torch.bfloat16, device="cuda")
    at = torch.from_numpy(rng.integers(0, n, rows)).cuda()
    logits.scatter_(1, at[:, None], 40.0)
    got = dw.sample_tokens(logits, uniforms(rng, rows), top_k=5)
    assert torch.equal(got.long(), at)


def test_graphs_streams_and_repeats():
    rng = np.random.default_rng(9)
    rows, n = 70, 30011
    logits, u = make(rng, rows, n, torch.bfloat16), uniforms(rng, rows)
    s = dict(top_k=torch.full((rows,), 500, dtype=torch.int32, device="cuda"), top_p=0.9, min_p=0.01)
    want = dw.sample_tokens(logits, u, **s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        dw.sample_tokens(logits, u, **s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = dw.sample_tokens(logits, u, **s)
    for turn in range(4):
        out.fill_(-9)
        torch.cuda.synchronize()
        g.replay()
        other = dw.sample_tokens(logits, u, **s)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)
    for stream in (side, side.cuda_stream):
        got = dw.sample_tokens(logits, u, stream=stream, **s)
        side.synchronize()
        assert torch.equal(got, want)
    u.copy_(uniforms(rng, rows))  # new random numbers reach a captured call
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, dw.sample_tokens(logits, u, **s))


def test_refusals():
    z, u = torch.zeros(4, 10, device="cuda"), torch.zeros(4, device="cuda")
    f = lambda q: torch.full((4,), q, device="cuda")  # noqa: E731
    for bad in (lambda: dw.sample_tokens(z.double(), u), lambda: dw.sample_tokens(z[0], u), lambda: dw.sample_tokens(z, u[:3]), lambda: dw.sample_tokens(z, u.double()),
                lambda: dw.sample_tokens(z, u.cpu()), lambda: dw.sample_tokens(z.cpu(), u), lambda: dw.sample_tokens(z.t(), u[:1].expand(10)),
                lambda: dw.sample_tokens(z, u, temperature=f(1.0).double()), lambda: dw.sample_tokens(z, u, top_k=f(1.0)),
                lambda: dw.sample_tokens(z, u, top_p=f(1.0)[:2]), lambda: dw.sample_tokens(z, u, min_p=f(1.0).cpu()),
                lambda: dw.sample_tokens(z, u, out=f(1.0)), lambda: dw.sample_tokens(z, u, out=torch.zeros(5, dtype=torch.int32, device="cuda")),
                lambda: dw.sample_tokens(torch.zeros(1, (1 << 19) + 1, device="cuda"), u[:1]), lambda: dw.sample_tokens(z[:, :0], u),
                lambda: dw.sample_tokens(z, u, out=u.view(torch.int32)), lambda: dw.sample_tokens(z.clone().requires_grad_(), u)):
        with pytest.raises((TypeError, ValueError, dw.ScanError)):
            bad()
    assert dw.sample_tokens(z[:0], u[:0]).shape == (0,)
    assert (dw.sample_tokens(z, u) == 0).all()
