"""The operators of a recurrent model with experts as a user's program calls them, with their plain forms.

Three groups: the gated linear recurrence (a prompt, a training step, a single token), tokens
sorted by expert and back with weights applied (forwards, and with every gradient), and
sampling with temperature, top-k, top-p and min-p from given random numbers.  ``listed()`` holds
the cases, ``draw`` more of the same ranges.  With ``own`` false, ``run`` computes a case from
elementary torch operations, in 32 bits but for sampling, whose sums meet borders (64 bits);
with it true, through the package's entry points.

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
        # one decoding step of 64 sequences whose states lie in a cache of slots
        dict(name="gate step 64", kind="gate_step", b=64, d=2560, t="bf16"),
        # one long prompt: few channels, so the rows have to be split
        dict(name="gate prompt 16384 f16", kind="gate", rows=16384, seqs=1, d=2048, t="f16"),
        # a batch of ragged prompts that continue from cached states
        dict(name="gate prompts ragged", kind="gate", rows=8191, seqs=9, d=4096, t="bf16"),
        # a training step: forward and every gradient
        dict(name="gate train 8x2048", kind="gate_train", b=8, l=2048, d=4096, t="bf16"),
        # one decoding step: 64 tokens, each to 8 of 64 experts
        dict(name="experts step 64", kind="experts", n=64, k=8, e=64, d=2048, t="bf16"),
        # the tokens of a batch of prompts
        dict(name="experts prompts 8192", kind="experts", n=8192, k=8, e=128, d=2048, t="bf16"),
        # a small training batch in 32 bits, rows that do not fill 16 bytes
        dict(name="experts train 1999 f32", kind="experts_train", n=1999, k=2, e=8, d=1002, t="f32"),
        # a training step: forward and every gradient
        dict(name="experts train 8192", kind="experts_train", n=8192, k=4, e=32, d=4096, t="bf16"),
        # one user's next token, one setting
        dict(name="sample 1x32000 f32", kind="sample", rows=1, v=32000, how="one", t="f32"),
        # a batch of users with settings of their own; an odd vocabulary
        dict(name="sample 64x50001 f32", kind="sample", rows=64, v=50001, how="own", t="f32"),
        # a large batch in 16 bits, where many logits are equal
        dict(name="sample 256x128000", kind="sample", rows=256, v=128000, how="own", t="bf16"),
        # drafts of a large batch: the whole distribution, temperature only
        dict(name="sample 512x131072 all", kind="sample", rows=512, v=131072, how="all", t="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gate_step", "gate", "gate_train", "experts", "experts_train", "sample", "sample"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "sample":
        rows = _log(rng, 1, 512)
        v = _log(rng, 256, min(200000, (1 << 25) // rows))
        return dict(kind=kind, rows=rows, v=v, how=rng.choice(["one", "own", "own", "all"]), t=t)
    d = rng.choice([_log(rng, 48, 5000), 64 * _log(rng, 2, 80)])
    if kind.startswith("experts"):
        k = rng.randint(1, 8)
        n = _log(rng, 1, min(16384, (1 << 26) // d // k))
        return dict(kind=kind, n=n, k=k, e=_log(rng, max(k, 4), 256), d=d, t=t)
    if kind == "gate_step":
        return dict(kind=kind, b=_log(rng, 1, 512), d=d, t=t)
    rows = _log(rng, 1, min(40000, (1 << 25) // d))
    if kind == "gate":
        return dict(kind=kind, rows=rows, seqs=min(rows, _log(rng, 1, 40)), d=d, t=t)
    b = rng.randint(1, 8)
    return dict(kind=kind, b=b, l=max(1, rows // b), d=d, t=t)


# ---------------------------------------------------------------------- inputs
class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 17)
        self.r = np.random.RandomState((int(seed) * 99991 + 3) % (1 << 32))

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

    def choices(self, n, k, e):
        """The k best experts of every token by scores that favour some experts, and their weights; in
        batches over 1000 tokens 2% are padding, which goes to no expert (-1)."""
        score = self.normal(n, e) + self.normal(e, scale=0.7)
        best, experts = score.topk(k, dim=1)
        experts = experts.int()
        if n > 1000:
            experts[self.uniform(n) < 0.02] = -1
        return experts, torch.softmax(best, 1)


def prepare(case, seed):
    c, m = case, _Maker(seed)
    t, kind = _T[c["t"]], c["kind"]
    if kind == "sample":
        rows, v = c["rows"], c["v"]
        # a few peaks above the rest; with settings of their own, some rows leave tokens out
        logits = m.normal(rows, v, scale=2.0) + 8.0 * (m.uniform(rows, v) < 20.0 / v)
        if c["how"] == "own":
            logits[1::3, 5:v // 2:7] = -math.inf
        s = dict(c, logits=logits.to(t), uniform=m.uniform(rows), temperature=0.8, top_k=0, top_p=1.0, min_p=0.0)
        if c["how"] == "one":
            s.update(top_k=50, top_p=0.95)
        elif c["how"] == "own":
            pick = lambda *of: torch.tensor(of, device="cuda")[torch.from_numpy(m.r.randint(0, len(of), rows)).cuda()]  # noqa: E731
            s.update(temperature=pick(0.0, 0.6, 0.8, 1.0, 1.3), top_k=pick(0, 20, 50, 1000).int(),
                     top_p=pick(0.8, 0.9, 0.95, 1.0), min_p=pick(0.0, 0.0, 0.02, 0.1))
        return s
    d = c["d"]
    if kind.startswith("experts"):
        n, k = c["n"], c["k"]
        experts, weights = m.choices(n, k, c["e"])
        s = dict(c, x=m.normal(n, d, t=t), experts=experts, weights=weights, y=m.normal(n * k, d, t=t))
        if kind == "experts_train":
            s.update(dout=m.normal(n, d, t=t), drows=m.normal(n * k, d, t=t))
        return s
    # rates whose factors at an open gate lie between 0.9 and 0.999, of an eighth of that at a closed one
    s = dict(c, rate=8.0 * torch.log(m.uniform(d, lo=0.9, hi=0.999)))
    lead = (c["b"],) if kind == "gate_step" else (c["rows"],) if kind == "gate" else (c["b"], c["l"])
    gates = m.normal(*lead, 2 * d, t=t)  # the two gates are the halves of a projection's output
    s.update(x=m.normal(*lead, d, t=t), decay_gate=gates[..., :d], input_gate=gates[..., d:])
    if kind == "gate_step":
        return dict(s, state=m.normal(c["b"] + 3, d), slots=m.slots(c["b"]))
    if kind == "gate":
        return dict(s, offsets=m.offsets(c["rows"], c["seqs"]), initial=m.normal(c["seqs"], d))
    return dict(s, dy=m.normal(*lead, d, t=t))


# ---------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _own(state, state["kind"])
    return _PLAIN[state["kind"]](state)


def _own(s, kind):
    import device_wide_prefix_tile_amd as dw

    if kind == "sample":
        return dw.sample_tokens(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                min_p=s["min_p"])
    if kind.startswith("experts"):
        plan = dw.expert_split(s["experts"], s["e"])
        rows = dw.expert_dispatch(s["x"], plan)
        out = dw.expert_combine(s["y"], plan, s["weights"])
        if kind == "experts":
            return plan.offsets, plan.places, plan.source, rows, out
        g = dw.expert_combine_grad(s["dout"], s["y"], plan, s["weights"])
        dx = dw.expert_dispatch_grad(s["drows"], plan)
        return plan.offsets, plan.places, plan.source, rows, out, g.dy, g.dweights, dx
    args = (s["x"], s["decay_gate"], s["input_gate"], s["rate"])
    if kind == "gate_step":
        return dw.gated_scan_step(*args, s["state"], slots=s["slots"]), s["state"]
    if kind == "gate":
        return dw.gated_scan(*args, seq_offsets=s["offsets"], initial_state=s["initial"], final_state=True)
    y, saved = dw.gated_scan(*args, save_for_grad=True)
    g = dw.gated_scan_grad(s["dy"], *args, saved=saved)
    return y, g.dx, g.ddecay_gate, g.dinput_gate, g.drate


# ---------------------------------------------------------------------- plain forms
def _gates(s, lead):
    """Both gates, the factor a, and the weight sqrt(1 - a^2) of the input."""
    r = torch.sigmoid(s["decay_gate"].flatten(0, lead).float())
    i = torch.sigmoid(s["input_gate"].flatten(0, lead).float())
    log_a = s["rate"] * r
    return r, i, torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t over dim 0, by composing the maps of spans that double."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], a[span:] * b[:-span] + b[span:]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _gate(s):
    x, off = s["x"].float(), s["offsets"].long()
    r, i, a, w = _gates(s, 0)
    b = w * i * x
    seq = torch.searchsorted(off[1:], torch.arange(x.shape[0], device="cuda"), right=True)
    first = torch.arange(x.shape[0], device="cuda") == off[seq]
    b[first] += a[first] * s["initial"][seq[first]]
    a = torch.where(first[:, None], 0.0, a)
    h = _recurrence(a, b)
    some = (off[1:] > off[:-1])[:, None]
    return h.to(s["x"].dtype), torch.where(some, h[(off[1:] - 1).clamp(min=0)], s["initial"])


def _gate_train(s):
    t, shape = s["x"].dtype, s["x"].shape
    x, dy = s["x"].flatten(0, 1).float(), s["dy"].flatten(0, 1).float()
    r, i, a, w = _gates(s, 1)
    first = torch.arange(x.shape[0], device="cuda") % s["l"] == 0
    past = torch.where(first[:, None], 0.0, a)
    h = _recurrence(past, w * i * x)
    dh = _recurrence(torch.cat([past[1:], torch.zeros_like(a[:1])]).flip(0), dy.flip(0)).flip(0)
    dlog = dh * (past * torch.cat([torch.zeros_like(h[:1]), h[:-1]]) - i * x * a * a / w)
    out = (h, dh * w * i, dlog * s["rate"] * r * (1 - r), dh * w * x * i * (1 - i))
    return tuple(v.to(t).view(shape) for v in out) + ((dlog * r).sum(0),)


def _gate_step(s):
    at = s["slots"].long()
    r, i, a, w = _gates(s, 0)
    h = a * s["state"][at] + w * i * s["x"].float()
    s["state"][at] = h
    return h.to(s["x"].dtype), s["state"]


def _split(s):
    """Counts by comparison: the place of a choice is the choices of smaller experts and the earlier ones of its own."""
    flat, e = s["experts"].flatten().long(), s["e"]
    of = (flat[:, None] == torch.arange(e, device="cuda")).int()
    count = of.sum(0)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    inside = (flat >= 0) & (flat < e)
    place = (offsets[:-1] + of.cumsum(0) - 1).gather(1, flat.clamp(0, e - 1)[:, None])[:, 0]
    source = torch.full_like(flat, -1)
    source[place[inside]] = torch.arange(flat.numel(), device="cuda")[inside]
    return offsets.int(), torch.where(inside, place, -1).int().view_as(s["experts"]), source.int()


def _from_places(y, places):
    """The row of every choice in 32 bits (n, k, D), zero where it has none."""
    return torch.where((places >= 0)[..., None], y.float()[places.long().clamp(min=0)], 0.0)


def _to_places(values, places, t):
    """Rows (n, k, D) at their places, zero where no choice leads."""
    out = torch.zeros(places.numel(), values.shape[-1], dtype=t, device="cuda")
    out[places[places >= 0].long()] = values[places >= 0].to(t)
    return out


def _experts(s):
    t = s["x"].dtype
    offsets, places, source = _split(s)
    rows = _to_places(s["x"][:, None].expand(-1, s["k"], -1), places, t)
    at = _from_places(s["y"], places)
    out = (at * s["weights"][..., None]).sum(1).to(t)
    if s["kind"] == "experts":
        return offsets, places, source, rows, out
    dout = s["dout"].float()[:, None]
    dy = _to_places(dout * s["weights"][..., None], places, t)
    dx = _from_places(s["drows"], places).sum(1).to(t)
    return offsets, places, source, rows, out, dy, (at * dout).sum(-1), dx


def _column(s, name, t):
    v = s[name]
    return v.to(t)[:, None] if torch.is_tensor(v) else torch.full((s["rows"], 1), v, dtype=t, device="cuda")


def _sample(s):
    """Tokens by falling logit, equal ones by index: top-k, top-p and min-p each keep a first part of them.  What
    is kept is summed up in the order of the indices."""
    logits, v = s["logits"].double(), s["v"]
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    temperature, top_k = _column(s, "temperature", torch.float64), _column(s, "top_k", torch.int64)
    greedy = temperature <= 0
    w = torch.exp((order.values - order.values[:, :1]) / torch.where(greedy, 1.0, temperature))
    rank = torch.arange(v, device="cuda")
    keep = (rank < torch.where(top_k > 0, top_k, v)) & (order.values > -math.inf)
    w = torch.where(keep, w, 0.0)
    before = torch.cumsum(w, 1) - w
    keep &= (before < _column(s, "top_p", torch.float64) * w.sum(1, keepdim=True)) & (w >= _column(s, "min_p", torch.float64) * w[:, :1])
    keep = torch.where(greedy, rank == 0, keep | (rank == 0))
    w = torch.zeros_like(w).scatter_(1, order.indices, torch.where(keep, w, 0.0))
    total = torch.cumsum(w, 1)
    return (total > s["uniform"].double()[:, None] * total[:, -1:]).int().argmax(1).int()


_PLAIN = dict(gate=_gate, gate_train=_gate_train, gate_step=_gate_step, experts=_experts, experts_train=_experts, sample=_sample)


# ---------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, kind = case, case["kind"]
    e = _SIZE[c["t"]]
    if kind == "sample":
        return dict(bytes=c["rows"] * (c["v"] * e + 8), flops=8 * c["rows"] * c["v"])
    d = c["d"]
    if kind.startswith("experts"):
        n, k = c["n"], c["k"]
        moved = e * d * (2 * n + 2 * n * k)  # x, the experts' rows; their results, the output
        flops = 2 * n * k * d
        if kind == "experts_train":
            moved += e * d * (2 * n + 3 * n * k)  # dout, results, their gradient; the rows' gradient, dx
            flops += 4 * n * k * d
        return dict(bytes=moved + 4 * n * k * (4 if kind == "experts" else 6), flops=flops)
    if kind == "gate_step":
        return dict(bytes=c["b"] * d * (4 * e + 8) + 4 * d, flops=20 * c["b"] * d)
    if kind == "gate":
        return dict(bytes=c["rows"] * d * 4 * e + 8 * c["seqs"] * d + 4 * d, flops=20 * c["rows"] * d)
    # forward: x, two gates, y; gradients: x, two gates, dy, dx, two gates'
    return dict(bytes=c["b"] * c["l"] * d * 11 * e + 12 * d, flops=60 * c["b"] * c["l"] * d)


# ---------------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "sample":
        return _exact_sample(s)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return _exact_experts(s) if s["kind"].startswith("experts") else _EXACT_GATE[s["kind"]](s)


def _exact_row(s, x, decay, gate, h):
    """One row of the recurrence, from the state h."""
    a = torch.exp(s["rate"] / (1 + torch.exp(-decay)))
    return a * h + torch.sqrt((1 - a) * (1 + a)) * x / (1 + torch.exp(-gate))


def _exact_gate_step(s):
    at = s["slots"].long()
    y = _exact_row(s, s["x"], s["decay_gate"], s["input_gate"], s["state"][at])
    s["state"][at] = y
    return y, s["state"]


def _exact_gate(s):
    o, y, last = s["offsets"].tolist(), torch.empty_like(s["x"]), []
    for q in range(s["seqs"]):
        h = s["initial"][q]
        for r in range(o[q], o[q + 1]):
            h = y[r] = _exact_row(s, s["x"][r], s["decay_gate"][r], s["input_gate"][r], h)
        last.append(h)
    return y, torch.stack(last)


def _exact_gate_train(s):
    """The recurrence row by row and its adjoint row by row backwards, all sequences at once."""
    x, l, rate = s["x"], s["l"], s["rate"]
    r, i = (1 / (1 + torch.exp(-s[q])) for q in ("decay_gate", "input_gate"))
    a = torch.exp(rate * r)
    w = torch.sqrt((1 - a) * (1 + a))
    h, y = torch.zeros_like(x[:, 0]), torch.empty_like(x)
    for q in range(l):
        h = y[:, q] = a[:, q] * h + w[:, q] * i[:, q] * x[:, q]
    dh = torch.empty_like(x)
    g = torch.zeros_like(h)
    for q in range(l - 1, -1, -1):
        g = dh[:, q] = s["dy"][:, q] + g
        g = g * a[:, q]
    before = torch.cat([torch.zeros_like(y[:, :1]), y[:, :-1]], 1)
    da = dh * (before - i * x * a / w)  # dw / da = -a / w
    dr = da * rate * a
    return y, dh * w * i, dr * r * (1 - r), dh * w * x * i * (1 - i), (da * a * r).sum((0, 1))


_EXACT_GATE = dict(gate=_exact_gate, gate_step=_exact_gate_step, gate_train=_exact_gate_train)


def _exact_experts(s):
    """Expert by expert: its choices in order, one run of rows each."""
    n, k, d = s["n"], s["k"], s["d"]
    flat = s["experts"].flatten()
    x, out, dw = s["x"], torch.zeros(n, d, dtype=torch.float64, device="cuda"), torch.zeros(n * k, dtype=torch.float64, device="cuda")
    rows, dy, dx = torch.zeros(n * k, d, dtype=torch.float64, device="cuda"), torch.zeros_like(s["y"]), torch.zeros_like(x)
    places, source, offsets = torch.full_like(flat, -1), torch.full_like(flat, -1), [0]
    weights = s["weights"].flatten()
    for e in range(s["e"]):
        of = torch.nonzero(flat == e)[:, 0]
        lo, hi = offsets[-1], offsets[-1] + of.numel()
        offsets.append(hi)
        token = of // k
        places[of] = torch.arange(lo, hi, dtype=torch.int32, device="cuda")
        source[lo:hi] = of.int()
        rows[lo:hi] = x[token]
        out.index_add_(0, token, s["y"][lo:hi] * weights[of, None])
        if s["kind"] == "experts_train":
            dy[lo:hi] = s["dout"][token] * weights[of, None]
            dw[of] = torch.linalg.vecdot(s["dout"][token], s["y"][lo:hi])
            dx.index_add_(0, token, s["drows"][lo:hi])
    got = torch.tensor(offsets, dtype=torch.int32, device="cuda"), places.view(n, k), source, rows, out
    if s["kind"] == "experts":
        return got
    dy[offsets[-1]:] = 0
    return got + (dy, dw.view(n, k), dx)


def _exact_sample(s):
    rows = s["rows"]
    wide = lambda q: np.broadcast_to(np.asarray(q.cpu() if torch.is_tensor(q) else q, dtype=np.float64), (rows,))  # noqa: E731
    temperature, top_k, top_p, min_p = (wide(s[q]) for q in ("temperature", "top_k", "top_p", "min_p"))
    u, tokens = s["uniform"].double().cpu().numpy(), []
    for r in range(rows):
        z = s["logits"][r].double().cpu().numpy()
        if temperature[r] <= 0:
            tokens.append(int(np.argmax(z)))
            continue
        p = np.exp((z - z.max()) / temperature[r])
        if top_k[r] > 0 or top_p[r] < 1:  # what the first k have, and their first part that reaches top_p of it
            order = np.argsort(-z, kind="stable")
            if top_k[r] > 0:
                order = order[:int(top_k[r])]
            most = np.concatenate([[0.0], np.cumsum(p[order])])
            left = order[(most[:-1] < top_p[r] * most[-1]) | (np.arange(order.size) == 0)]
            kept = np.zeros_like(p)
            kept[left] = p[left]
            p = kept
        p[p < min_p[r]] = 0
        run_up = np.cumsum(p)
        tokens.append(int(np.searchsorted(run_up, u[r] * run_up[-1], side="right")))
    return torch.tensor(tokens, dtype=torch.int32, device="cuda")
