"""Sampled tokens of whole batches against the definition in 64 bits, row by row and without a tolerance: a token may
differ only where the random number or the border of top-p lies within 2^-36 of another token's share.

Why 2^-36: a weight of the kernel is off by 2^-44 of itself at most (the exponent's product, 60 times 2^-53 for what
weighs 2^-60 and more; its polynomial 2^-44.6; a few roundings), a sum of n of them by log2(n) 2^-53 more; where weights
are added up as integers each is off by half a unit of 2^-(63 - log2 n), of n = 2^19 together by 2^-26 at the very
worst and by sqrt(n) / 2 units = 2^-35.5 of a sum of at least one in the mean square; the vocabulary here is 2^17
(2^-38.5).  A difference that the bound allows is met with a probability of 2^17 2^-35, 4e-6, per row."""
import pytest
import torch

import device_wide_prefix_tile_amd as dw

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEAR = 2.0 ** -36


def make(g, rows, n, t, std=2.0):
    z = torch.randn(rows, n, generator=g, device="cuda") * std + 8.0 * (torch.rand(rows, n, generator=g, device="cuda") < 20.0 / n)
    return z.to(t), torch.rand(rows, generator=g, device="cuda")


def weights(logits, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """The kept weights (rows, n) in 64 bits, by index."""
    z = logits.double()
    z = torch.where(z.isnan(), -float("inf"), z)
    w = torch.exp((z - z.amax(1, keepdim=True)) / temperature)
    if top_k > 0 or top_p < 1.0:
        order = torch.sort(z, dim=1, descending=True, stable=True).indices
        s = w.gather(1, order)
        if top_k > 0:
            s[:, top_k:] = 0
        before = torch.cumsum(s, 1) - s
        keep = before < top_p * s.sum(1, keepdim=True) if top_p < 1.0 else torch.ones_like(s, dtype=torch.bool)
        keep[:, 0] = True
        w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, s, 0.0))
    return torch.where(w >= min_p, w, 0.0)


def tokens(w, u):
    run = torch.cumsum(w, 1)
    return (run > u.double()[:, None] * run[:, -1:]).int().argmax(1).int()


def differing(logits, u, got, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(rows whose token is not the definition's, those of them that a border nearer than NEAR does not explain)"""
    s = (temperature, top_k)
    w = weights(logits, *s, top_p, min_p)
    want = tokens(w, u)
    bad = torch.nonzero(got != want)[:, 0]
    if not bad.numel():
        return 0, 0
    explained = torch.zeros(bad.numel(), dtype=torch.bool, device="cuda")
    for p in (top_p, top_p - NEAR, top_p + NEAR) if top_p < 1.0 else (top_p,):
        w = weights(logits[bad], *s, p, min_p)
        for v in (-NEAR, 0.0, NEAR):
            explained |= tokens(w, u[bad].double() + v) == got[bad]
    return bad.numel(), int((~explained).sum())


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("s", [dict(temperature=0.8), dict(temperature=1.0, top_p=0.95), dict(temperature=1.3, top_p=0.8, min_p=1e-4)],
                         ids=["all", "top-p", "top-p min-p"])
def test_every_token_of_large_batches(t, s):
    g = torch.Generator(device="cuda").manual_seed(len(t) + len(s))
    off = unexplained = 0
    for _ in range(8):
        logits, u = make(g, 512, 131072, T[t])
        got = dw.sample_tokens(logits, u, **s)
        d = differing(logits, u, got, **s)
        off, unexplained = off + d[0], unexplained + d[1]
    # 4096 rows: 0.02 expected
    assert unexplained == 0 and off <= 1, "%d of 4096 tokens differ, %d without a border beside them" % (off, unexplained)


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("n,s", [(30000, dict(temperature=2.0, top_k=700)), (2000, dict(temperature=3.0, top_k=1900, top_p=0.97)),
                                 (50001, dict(temperature=1.5, top_k=5000, top_p=0.9)), (128000, dict(temperature=2.0, top_k=1000))])
def test_every_token_with_top_k(t, n, s):
    g = torch.Generator(device="cuda").manual_seed(n)
    off = unexplained = 0
    for _ in range(2):
        logits, u = make(g, 512, n, T[t])
        d = differing(logits, u, dw.sample_tokens(logits, u, **s), **s)
        off, unexplained = off + d[0], unexplained + d[1]
    assert unexplained == 0 and off <= 1


@pytest.mark.parametrize("t", list(T))
def test_the_smallest_weights_are_weights(t):
    """A random number of 0 takes the first kept token that weighs anything, in every way a row may take: a token of a
    weight of e^-80 and more is kept, one of minus infinity is not there."""
    for n, at in ((5, 1), (40, 1), (2048, 3), (5000, 2), (60000, 1)):
        z = torch.zeros(4, n, device="cuda")
        z[:, :at] = -float("inf")
        z[:, at] = torch.tensor([-30.0, -45.0, -60.0, -80.0], device="cuda")
        u = torch.zeros(4, device="cuda")
        for s in (dict(), dict(top_k=n - at), dict(min_p=1e-36), dict(top_k=n - at, min_p=1e-36)):
            got = dw.sample_tokens(z.to(T[t]), u, **s)
            assert (got == at).all(), (n, s, got)
    # beyond the range of 32 bits: e^-600
    z = torch.zeros(3, 3000, device="cuda")
    z[:, 0] = -600.0
    u = torch.tensor([0.0, 2.0 ** -24, 0.5], device="cuda")
    for s in (dict(), dict(top_k=3000 - 1), dict(top_k=3000)):
        got = dw.sample_tokens(z.to(T[t]), u, **s).tolist()
        assert got[0] == (1 if s.get("top_k") == 2999 else 0) and got[1] == 1, (s, got)
