"""The sequence operators as a user's program calls them, with their plain forms.

Four operators: embedding lookup, its gradient, the short causal convolution and the
selective state-space scan (each of the last two as a prompt, a training step and a single
token).  ``listed()`` holds the cases, ``draw`` more of the same ranges.  With ``own`` false,
``run`` computes a case from elementary torch operations in 32 bits; with it true, through
the package's entry points.

Rows are flat and channels come last: a batch of B sequences of length L is (B, L, D), ragged
prompts are (rows, D) with the sequences' offsets.
"""
import math

import numpy as np
import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a batch: 64 rows of a large table
        dict(name="lookup 64 tokens", kind="lookup", n=64, v=50000, d=2048, t="bf16"),
        # the tokens of a batch of prompts
        dict(name="lookup 16384 tokens", kind="lookup", n=16384, v=32000, d=2560, t="bf16"),
        # a small training batch, gradient kept in 32 bits
        dict(name="table grad 4096 f32", kind="grad", n=4096, v=32000, d=1024, t="f32"),
        # a training batch with the skew of natural text and padded positions
        dict(name="table grad 65536", kind="grad", n=65536, v=50000, d=2048, t="bf16"),
        # one decoding step: the convolution of 64 sequences whose states lie in a cache of slots
        dict(name="conv step 64", kind="conv_step", b=64, d=4096, k=4, t="bf16"),
        # a batch of ragged prompts that continue from cached states
        dict(name="conv prompts ragged", kind="conv", rows=8191, seqs=9, d=4096, k=4, t="bf16"),
        # a training step: forward and gradients
        dict(name="conv train 8x2048", kind="conv_train", b=8, l=2048, d=4096, k=4, t="bf16"),
        # one decoding step of a small and of a large batch
        dict(name="scan step 16", kind="scan_step", b=16, d=2048, n=16, g=1, t="bf16"),
        dict(name="scan step 256", kind="scan_step", b=256, d=4096, n=16, g=1, t="bf16"),
        # one long prompt: few channels, so the rows have to be split
        dict(name="scan prompt 16384", kind="scan", rows=16384, seqs=1, d=2048, n=16, g=1, t="bf16"),
        # ragged prompts with two groups of B and C that share them among their channels
        dict(name="scan prompts ragged f16", kind="scan", rows=6001, seqs=12, d=4096, n=16, g=2, t="f16"),
        # a training step: forward and every gradient
        dict(name="scan train 4x2048", kind="scan_train", b=4, l=2048, d=4096, n=16, g=1, t="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["lookup", "grad", "conv_step", "conv", "conv_train", "scan_step", "scan", "scan_train"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("lookup", "grad"):
        d = rng.choice([_log(rng, 64, 4096), 8 * _log(rng, 8, 512)])
        return dict(kind=kind, n=_log(rng, 1, min(65536, (1 << 27) // d)), v=_log(rng, 256, 100000), d=d, t=t)
    d = rng.choice([_log(rng, 48, 5000), 64 * _log(rng, 2, 80)])
    if kind == "conv_step":
        return dict(kind=kind, b=_log(rng, 1, 512), d=d, k=rng.randint(2, 4), t=t)
    if kind == "conv":
        rows = _log(rng, 1, min(30000, (1 << 25) // d))
        return dict(kind=kind, rows=rows, seqs=min(rows, _log(rng, 1, 40)), d=d, k=rng.randint(2, 4), t=t)
    if kind == "conv_train":
        b = rng.randint(1, 9)
        return dict(kind=kind, b=b, l=_log(rng, 1, min(40000, (1 << 25) // d // b)), d=d, k=rng.randint(2, 4), t=t)
    n = rng.choice([16, 16, 16, rng.randint(4, 64)])
    g = rng.choice([1, 1, 2, 4])
    d = max(g, d // g * g)
    if kind == "scan_step":
        return dict(kind=kind, b=_log(rng, 1, min(512, (1 << 25) // d // n)), d=d, n=n, g=g, t=t)
    rows = _log(rng, 1, min(40000, (1 << 28) // d // n))
    if kind == "scan":
        return dict(kind=kind, rows=rows, seqs=min(rows, _log(rng, 1, 40)), d=d, n=n, g=g, t=t)
    b = rng.randint(1, 8)
    return dict(kind=kind, b=b, l=max(1, rows // b), d=d, n=n, g=g, t=t)


# ---------------------------------------------------------------------- inputs
class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
        self.r = np.random.RandomState((int(seed) * 104729 + 5) % (1 << 32))

    def normal(self, *shape, t=torch.float32, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale + mean).to(t)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def offsets(self, rows, seqs):
        """Ragged lengths that add up to `rows`; with three sequences or more, one of them is empty."""
        cut = np.sort(self.r.randint(0, rows + 1, seqs - 1))
        o = np.concatenate([[0], cut, [rows]]).astype(np.int32)
        if seqs > 2:
            o[2] = o[1]
        return torch.from_numpy(o).cuda()

    def slots(self, b):
        return torch.from_numpy(self.r.permutation(b + 3)[:b].astype(np.int32)).cuda()

    def tokens(self, n, v):
        """Frequencies that fall as 1 / rank, spread over the table; 2% padding (-1) in batches over 1000."""
        u = torch.rand(n, generator=self.g, device="cuda", dtype=torch.float64)
        rank = torch.exp(u * math.log(v + 1.0)).long().clamp_(1, v) - 1
        tok = rank * 48271 % v if math.gcd(48271, v) == 1 else rank
        if n > 1000:
            tok[torch.rand(n, generator=self.g, device="cuda") < 0.02] = -1
        return tok.int()


def prepare(case, seed):
    c, m = case, _Maker(seed)
    t, kind, d = _T[c["t"]], c["kind"], c["d"]
    if kind == "lookup":
        return dict(c, tokens=m.tokens(c["n"], c["v"]), table=m.normal(c["v"], d, t=t, scale=0.02), scale=math.sqrt(d))
    if kind == "grad":
        return dict(c, tokens=m.tokens(c["n"], c["v"]), dout=m.normal(c["n"], d, t=t), scale=math.sqrt(d))
    if kind.startswith("conv"):
        k = c["k"]
        s = dict(c, weight=m.normal(d, k, t=t, scale=k ** -0.5), bias=m.normal(d, t=t, scale=0.1))
        if kind == "conv_step":
            return dict(s, x=m.normal(c["b"], d, t=t), state=m.normal(c["b"] + 3, k - 1, d, t=t), slots=m.slots(c["b"]))
        if kind == "conv":  # x is one half of a projection's output
            return dict(s, x=m.normal(c["rows"], 2 * d, t=t)[:, :d], offsets=m.offsets(c["rows"], c["seqs"]),
                        initial=m.normal(c["seqs"], k - 1, d, t=t))
        return dict(s, x=m.normal(c["b"], c["l"], 2 * d, t=t)[..., :d], dy=m.normal(c["b"], c["l"], d, t=t))
    n, g = c["n"], c["g"]
    dt = torch.exp(m.uniform(d, lo=math.log(1e-3), hi=math.log(0.1)))
    s = dict(c, A=-torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * m.uniform(d, n, lo=0.9, hi=1.1),
             D=m.normal(d, mean=1.0, scale=0.1), delta_bias=torch.log(torch.expm1(dt)))
    lead = (c["b"],) if kind == "scan_step" else (c["rows"],) if kind == "scan" else (c["b"], c["l"])
    bc = m.normal(*lead, 2 * g * n, t=t)  # B and C are the two halves of a projection's output
    s.update(x=m.normal(*lead, d, t=t), delta=m.normal(*lead, d, t=t, scale=0.5), z=m.normal(*lead, 2 * d, t=t)[..., d:],
             B=bc[..., :g * n].unflatten(-1, (g, n)), C=bc[..., g * n:].unflatten(-1, (g, n)))
    if kind == "scan_step":
        return dict(s, state=m.normal(c["b"] + 3, d, n), slots=m.slots(c["b"]))
    if kind == "scan":
        return dict(s, offsets=m.offsets(c["rows"], c["seqs"]), initial=m.normal(c["seqs"], d, n))
    return dict(s, dy=m.normal(*lead, d, t=t))


# ---------------------------------------------------------------------- one pass
def run(state):
    s, kind = state, state["kind"]
    if own:
        return _own(s, kind)
    return _PLAIN[kind](s)


def _own(s, kind):
    import device_wide_prefix_tile_amd as dw

    if kind == "lookup":
        return dw.embedding_lookup(s["tokens"], s["table"], scale=s["scale"])
    if kind == "grad":
        return dw.embedding_grad(s["tokens"], s["dout"], s["v"], scale=s["scale"])
    if kind == "conv_step":
        y = dw.causal_conv1d_step(s["x"], s["state"], s["weight"], s["bias"], activation="silu", slots=s["slots"])
        return y, s["state"]
    if kind == "conv":
        return dw.causal_conv1d(s["x"], s["weight"], s["bias"], activation="silu", seq_offsets=s["offsets"],
                                initial_state=s["initial"], final_state=True)
    if kind == "conv_train":
        y = dw.causal_conv1d(s["x"], s["weight"], s["bias"], activation="silu")
        g = dw.causal_conv1d_grad(s["dy"], s["x"], s["weight"], s["bias"], activation="silu")
        return y, g.dx, g.dweight, g.dbias
    args = (s["x"], s["delta"], s["A"], s["B"], s["C"])
    kw = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], delta_softplus=True)
    if kind == "scan_step":
        return dw.selective_scan_step(*args, s["state"], slots=s["slots"], **kw), s["state"]
    if kind == "scan":
        return dw.selective_scan(*args, seq_offsets=s["offsets"], initial_state=s["initial"], final_state=True, **kw)
    y, saved = dw.selective_scan(*args, save_for_grad=True, **kw)
    g = dw.selective_scan_grad(s["dy"], *args, saved=saved, **kw)
    return y, g.dx, g.ddelta, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddelta_bias


# ---------------------------------------------------------------------- plain forms
def _lookup(s):
    tok = s["tokens"].long()
    inside = (tok >= 0) & (tok < s["v"])
    rows = s["table"][tok.clamp(0, s["v"] - 1)].float() * s["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(s["table"].dtype)


def _grad(s):
    tok = s["tokens"].long()
    inside = (tok >= 0) & (tok < s["v"])
    total = torch.zeros(s["v"] + 1, s["d"], device=tok.device)
    total.index_add_(0, torch.where(inside, tok, s["v"]), s["dout"].float())
    return (total[:-1] * s["scale"]).to(s["dout"].dtype)


def _silu(u):
    return u * torch.sigmoid(u)


def _dsilu(u):
    sig = torch.sigmoid(u)
    return sig * (1 + u * (1 - sig))


def _sequences(s, rows):
    """Offsets of the sequences, and each row's sequence."""
    if "offsets" in s:
        off = s["offsets"].long()
    else:
        off = torch.arange(s["b"] + 1, device="cuda") * s["l"]
    return off, torch.searchsorted(off[1:], torch.arange(rows, device="cuda"), right=True)


def _taps(x, initial, off, seq, k, pos):
    """(len(pos), k, d): the k inputs that end at position pos of sequence seq, earlier ones from the initial state."""
    nseq = off.numel() - 1
    source = torch.cat([x, initial.reshape(nseq * (k - 1), -1)])
    at = pos[:, None] - (k - 1) + torch.arange(k, device=x.device)
    first = x.shape[0] + (seq * (k - 1) + (k - 1))[:, None]
    return source[torch.where(at >= off[seq][:, None], at, first + at - off[seq][:, None])]


def _conv_parts(s):
    x = s["x"].flatten(0, -2).float()
    off, seq = _sequences(s, x.shape[0])
    k = s["k"]
    initial = s["initial"].float() if "initial" in s else torch.zeros(off.numel() - 1, k - 1, s["d"], device="cuda")
    taps = _taps(x, initial, off, seq, k, torch.arange(x.shape[0], device="cuda"))
    w = s["weight"].float()
    return x, off, seq, initial, taps, w, (taps * w.t()).sum(1) + s["bias"].float()


def _conv(s):
    x, off, seq, initial, taps, w, u = _conv_parts(s)
    nseq, t = off.numel() - 1, s["x"].dtype
    last = _taps(x, initial, off, torch.arange(nseq, device="cuda"), s["k"], off[1:] - 1)
    return _silu(u).to(t), last[:, 1:].to(t)


def _conv_train(s):
    x, off, seq, initial, taps, w, u = _conv_parts(s)
    k, t = s["k"], s["x"].dtype
    g = s["dy"].flatten(0, -2).float() * _dsilu(u)
    # row t goes into the outputs t .. t + k - 1 of its sequence
    at = torch.arange(x.shape[0], device="cuda")[:, None] + torch.arange(k - 1, -1, -1, device="cuda")
    at = torch.where(at < off[seq + 1][:, None], at, x.shape[0])
    dx = (torch.cat([g, g.new_zeros(1, s["d"])])[at] * w.t()).sum(1)
    return (_silu(u).to(t).view_as(s["dy"]), dx.to(t).view_as(s["dy"]), (g[:, None] * taps).sum(0).t().contiguous(),
            g.sum(0))


def _conv_step(s):
    at = s["slots"].long()
    taps = torch.cat([s["state"][at], s["x"][:, None]], 1)
    s["state"][at] = taps[:, 1:]
    u = (taps.float() * s["weight"].float().t()).sum(1) + s["bias"].float()
    return _silu(u).to(s["x"].dtype), s["state"]


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t over dim 0, by composing the maps of spans that double."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], a[span:] * b[:-span] + b[span:]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _spread(bc, d):
    """(rows, g, n) in 32 bits as (rows, d, n): each group's values for all of its channels."""
    return bc.float().repeat_interleave(d // bc.shape[-2], -2)


def _scan_parts(s):
    d = s["d"]
    x, z = s["x"].flatten(0, -2).float(), s["z"].flatten(0, -2).float()
    raw = s["delta"].flatten(0, -2).float() + s["delta_bias"]
    delta = _softplus(raw)
    B, C = _spread(s["B"].flatten(0, -3), d), _spread(s["C"].flatten(0, -3), d)
    off, seq = _sequences(s, x.shape[0])
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * x)[..., None] * B
    heads = torch.zeros(x.shape[0] + 1, dtype=torch.bool, device="cuda")
    heads[off[:-1]] = True
    heads = heads[:-1]
    if "initial" in s:
        b[heads] += a[heads] * s["initial"][seq[heads]]
    a[heads] = 0.0
    return x, z, raw, delta, B, C, off, heads, a, b


def _scan(s):
    x, z, raw, delta, B, C, off, heads, a, b = _scan_parts(s)
    h = _recurrence(a, b)
    y = ((C * h).sum(-1) + s["D"] * x) * _silu(z)
    some = (off[1:] > off[:-1])[:, None, None]
    return y.to(s["x"].dtype), torch.where(some, h[(off[1:] - 1).clamp(min=0)], s["initial"])


def _scan_train(s):
    x, z, raw, delta, B, C, off, heads, a, b = _scan_parts(s)
    t, shape, (g, n) = s["x"].dtype, s["x"].shape, s["B"].shape[-2:]
    h = _recurrence(a, b)
    del b
    v = (C * h).sum(-1) + s["D"] * x
    gate = _silu(z)
    dy = s["dy"].flatten(0, -2).float()
    dv = dy * gate
    later = torch.cat([a[1:], torch.zeros_like(a[:1])]).flip(0)
    dh = _recurrence(later, (dv[..., None] * C).flip(0)).flip(0)
    del later
    rows = x.shape[0]
    dC = (dv[..., None] * h).view(rows, g, -1, n).sum(2)
    dB = (dh * (delta * x)[..., None]).view(rows, g, -1, n).sum(2)
    before = a * torch.cat([torch.zeros_like(h[:1]), h[:-1]])  # a is zero where a sequence begins
    del h, a
    dhB = (dh * B).sum(-1)
    p = dh * before
    ddelta = (p * s["A"]).sum(-1) + dhB * x
    dpre = ddelta * torch.where(raw > 20, 1.0, torch.sigmoid(raw))
    return ((v * gate).to(t).view(shape), (dv * s["D"] + delta * dhB).to(t).view(shape), dpre.to(t).view(shape),
            (p * delta[..., None]).sum(0), dB.to(t).view(s["B"].shape), dC.to(t).view(s["C"].shape), (dv * x).sum(0),
            (dy * v * _dsilu(z)).to(t).view(shape), dpre.sum(0))


def _scan_step(s):
    at, d, x = s["slots"].long(), s["d"], s["x"].float()
    delta = _softplus(s["delta"].float() + s["delta_bias"])
    h = torch.exp(delta[..., None] * s["A"]) * s["state"][at] + (delta * x)[..., None] * _spread(s["B"], d)
    s["state"][at] = h
    y = ((h * _spread(s["C"], d)).sum(-1) + s["D"] * x) * _silu(s["z"].float())
    return y.to(s["x"].dtype), s["state"]


_PLAIN = dict(lookup=_lookup, grad=_grad, conv=_conv, conv_train=_conv_train, conv_step=_conv_step, scan=_scan,
              scan_train=_scan_train, scan_step=_scan_step)


# ---------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    e, d, kind = _SIZE[c["t"]], c["d"], c["kind"]
    if kind == "lookup":
        return dict(bytes=4 * c["n"] + 2 * e * d * c["n"], flops=d * c["n"])
    if kind == "grad":
        return dict(bytes=4 * c["n"] + e * d * (c["n"] + c["v"]), flops=2 * d * c["n"])
    if kind == "conv_step":
        k, b = c["k"], c["b"]
        return dict(bytes=e * d * (b * (2 + 2 * (k - 1)) + k + 1) + 4 * b, flops=b * d * (2 * k + 4))
    if kind == "conv":
        k = c["k"]
        return dict(bytes=e * d * (2 * c["rows"] + 2 * c["seqs"] * (k - 1) + k + 1), flops=c["rows"] * d * (2 * k + 4))
    if kind == "conv_train":
        k, rows = c["k"], c["b"] * c["l"]
        # forward: x, y; gradients: x, dy, dx
        return dict(bytes=e * d * (5 * rows + 2 * (k + 1)) + 4 * d * (k + 1), flops=rows * d * (8 * k + 14))
    n, g = c["n"], c["g"]
    params = 4 * d * (n + 2)
    if kind == "scan_step":
        b = c["b"]
        return dict(bytes=8 * b * d * n + e * b * (4 * d + 2 * g * n) + params + 4 * b, flops=b * d * (7 * n + 12))
    rows = c["rows"] if kind == "scan" else c["b"] * c["l"]
    if kind == "scan":
        return dict(bytes=e * rows * (4 * d + 2 * g * n) + 8 * c["seqs"] * d * n + params, flops=rows * d * (7 * n + 12))
    # forward: x, delta, z, B, C, y; gradients: x, delta, z, dy, B, C, dx, ddelta, dz, dB, dC
    return dict(bytes=e * rows * (11 * d + 6 * g * n) + 3 * params, flops=rows * d * (7 * n + 12 + 24 * n + 30))


# ---------------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    kind, d = s["kind"], s["d"]
    if kind == "lookup":
        zero = s["table"].new_zeros(1, d)
        tok = s["tokens"].long()
        return s["scale"] * torch.cat([s["table"], zero])[torch.where((tok < 0) | (tok >= s["v"]), s["v"], tok)]
    if kind == "grad":
        tok = s["tokens"].long()
        tok, order = torch.sort(torch.where((tok < 0) | (tok >= s["v"]), s["v"], tok))
        sums = torch.cat([s["dout"].new_zeros(1, d), torch.cumsum(s["dout"][order], 0)])
        edge = torch.searchsorted(tok, torch.arange(s["v"] + 1, device=tok.device))
        return s["scale"] * (sums[edge[1:]] - sums[edge[:-1]])
    if kind == "conv_step":
        y = []
        for i, at in enumerate(s["slots"].tolist()):
            window = torch.cat([s["state"][at], s["x"][i:i + 1]])
            u = s["bias"] + sum(s["weight"][:, j] * window[j] for j in range(s["k"]))
            y.append(u / (1 + torch.exp(-u)))
            s["state"][at] = window[1:]
        return torch.stack(y), s["state"]
    if kind == "scan_step":
        y = []
        for i, at in enumerate(s["slots"].tolist()):
            y.append(_exact_scan_row(s, s["x"][i], s["delta"][i], s["z"][i], s["B"][i], s["C"][i], s["state"][at]))
        return torch.stack(y), s["state"]
    if kind == "conv":
        o, y, fin = s["offsets"].tolist(), torch.empty(s["rows"], d, dtype=torch.float64, device="cuda"), []
        for i in range(s["seqs"]):
            whole = torch.cat([s["initial"][i], s["x"][o[i]:o[i + 1]]])
            u = s["bias"] + (whole.unfold(0, s["k"], 1) * s["weight"]).sum(-1) if o[i + 1] > o[i] else whole[:0]
            y[o[i]:o[i + 1]] = u / (1 + torch.exp(-u))
            fin.append(whole[whole.shape[0] - (s["k"] - 1):])
        return y, torch.stack(fin)
    if kind == "conv_train":
        with torch.enable_grad():
            x, w, b = (s[q].detach().clone().requires_grad_() for q in ("x", "weight", "bias"))
            u = b + (torch.nn.functional.pad(x, (0, 0, s["k"] - 1, 0)).unfold(1, s["k"], 1) * w).sum(-1)
            y = u / (1 + torch.exp(-u))
            return (y.detach(),) + torch.autograd.grad(y, (x, w, b), s["dy"])
    if kind == "scan":
        o, y, fin = s["offsets"].tolist(), torch.empty(s["rows"], d, dtype=torch.float64, device="cuda"), []
        for i in range(s["seqs"]):
            h = s["initial"][i].clone()
            for r in range(o[i], o[i + 1]):
                y[r] = _exact_scan_row(s, s["x"][r], s["delta"][r], s["z"][r], s["B"][r], s["C"][r], h)
            fin.append(h)
        return y, torch.stack(fin)
    return _exact_scan_train(s)


def _exact_scan_row(s, x, delta, z, B, C, h):
    """One row: the state h is updated in place."""
    per = s["d"] // s["g"]
    dt = torch.logaddexp(delta + s["delta_bias"], torch.zeros_like(delta))
    h.mul_(torch.exp(dt[:, None] * s["A"])).add_((dt * x)[:, None] * B.repeat_interleave(per, 0))
    return (torch.linalg.vecdot(h, C.repeat_interleave(per, 0)) + s["D"] * x) * z / (1 + torch.exp(-z))


def _exact_scan_train(s):
    """The recurrence row by row and its adjoint row by row backwards, all sequences at once."""
    b, l, d = s["x"].shape
    g, n, per = s["g"], s["n"], d // s["g"]
    x, z, dy, A = s["x"], s["z"], s["dy"], s["A"]
    raw = s["delta"] + s["delta_bias"]
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    wide = lambda v: v.repeat_interleave(per, 1)  # noqa: E731
    hs = torch.empty(l + 1, b, d, n, dtype=torch.float64, device="cuda")
    hs[0] = 0
    for t in range(l):
        torch.addcmul(torch.exp(dt[:, t, :, None] * A) * hs[t], (dt[:, t] * x[:, t])[..., None], wide(s["B"][:, t]), out=hs[t + 1])
    out = {k: torch.empty_like(x) for k in ("y", "dx", "ddt", "dz")}
    dB, dC, dA = torch.empty_like(s["B"]), torch.empty_like(s["C"]), torch.zeros_like(A)
    sig = 1 / (1 + torch.exp(-z))
    dh = torch.zeros_like(hs[0])
    for t in range(l - 1, -1, -1):
        Bt, Ct, xt, dtt = wide(s["B"][:, t]), wide(s["C"][:, t]), x[:, t], dt[:, t]
        v = (hs[t + 1] * Ct).sum(-1) + s["D"] * xt
        dv = dy[:, t] * z[:, t] * sig[:, t]
        out["y"][:, t] = v * z[:, t] * sig[:, t]
        out["dz"][:, t] = dy[:, t] * v * (sig[:, t] + z[:, t] * sig[:, t] * (1 - sig[:, t]))
        dh += dv[..., None] * Ct
        dC[:, t] = (dv[..., None] * hs[t + 1]).view(b, g, per, n).sum(2)
        dB[:, t] = ((dtt * xt)[..., None] * dh).view(b, g, per, n).sum(2)
        along = (dh * Bt).sum(-1)
        decay = torch.exp(dtt[..., None] * A)
        through = dh * decay * hs[t]
        out["dx"][:, t] = dv * s["D"] + dtt * along
        out["ddt"][:, t] = along * xt + (through * A).sum(-1)
        dA += (through * dtt[..., None]).sum(0)
        dh *= decay
    dD = (dy * z * sig * x).sum((0, 1))
    draw = out["ddt"] / (1 + torch.exp(-raw))
    return out["y"], out["dx"], draw, dA, dB, dC, dD, out["dz"], draw.sum((0, 1))
