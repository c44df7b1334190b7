"""The operators together as a recurrent model with experts runs them: embedding, convolution, gated recurrence, experts,
logits, next token; as a prompt, token by token, and a training pass."""
import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import sampling_reference as sr

pytestmark = pytest.mark.gpu

V, D, E, K = 300, 48, 6, 2


def randn(rng, *shape, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).float().cuda()


def params(rng):
    return dict(table=randn(rng, V, D, scale=0.5), w=randn(rng, D, 4, scale=0.5), b=randn(rng, D, scale=0.1), gates=randn(rng, D, 2 * D, scale=D ** -0.5),
                rate=-torch.from_numpy(np.exp(rng.uniform(np.log(0.01), np.log(2.0), D))).float().cuda(), router=randn(rng, D, E),
                experts=randn(rng, E, D, D, scale=D ** -0.5), head=randn(rng, D, V))


def experts(p, h, choice=None):
    """(output, plan, weights, dispatched rows, the experts' results)"""
    score, best = (h @ p["router"]).topk(K, dim=1)
    best = best.int() if choice is None else choice
    weights = torch.softmax(score, 1)
    plan = dw.expert_split(best, E)
    rows = dw.expert_dispatch(h, plan)
    y = torch.zeros_like(rows)
    ends = plan.offsets.tolist()
    for e in range(E):
        y[ends[e]:ends[e + 1]] = rows[ends[e]:ends[e + 1]] @ p["experts"][e]
    return dw.expert_combine(y, plan, weights), plan, weights, rows, y


def prompt(p, tokens, off, conv=None, state=None):
    e = dw.embedding_lookup(tokens, p["table"], scale=2.0)
    u, conv = dw.causal_conv1d(e, p["w"], p["b"], activation="silu", seq_offsets=off, initial_state=conv, final_state=True)
    gates = u @ p["gates"]
    h, state = dw.gated_scan(u, gates[:, :D], gates[:, D:], p["rate"], seq_offsets=off, initial_state=state, final_state=True)
    return experts(p, h)[0] @ p["head"], conv, state


def step(p, tokens, conv, state, slots):
    e = dw.embedding_lookup(tokens, p["table"], scale=2.0)
    u = dw.causal_conv1d_step(e, conv, p["w"], p["b"], activation="silu", slots=slots)
    gates = u @ p["gates"]
    h = dw.gated_scan_step(u, gates[:, :D], gates[:, D:], p["rate"], state, slots=slots)
    return experts(p, h)[0] @ p["head"]


def test_prompts_then_tokens():
    """Ragged prompts, then tokens drawn one by one from the logits and fed back, the states in slots: the logits are those
    of the whole sequences as prompts, up to 32-bit roundings of a hundred operations on values of their size."""
    rng = np.random.default_rng(1)
    p = params(rng)
    lengths, steps = [70, 1, 33], 6
    text = [rng.integers(0, V, n).astype(np.int32) for n in lengths]
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    off = dev(np.cumsum([0] + lengths))
    logits, conv, state = prompt(p, dev(np.concatenate(text)), off)
    slots = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    convs, states = torch.zeros(5, 3, D, device="cuda"), torch.zeros(5, D, device="cuda")
    convs[slots.long()], states[slots.long()] = conv, state
    last = logits[(off[1:] - 1).long()]
    setting = dict(temperature=torch.tensor([0.0, 0.8, 1.2], device="cuda"), top_k=torch.tensor([0, 40, 0], dtype=torch.int32, device="cuda"), top_p=0.9)
    for i in range(steps):
        u = torch.from_numpy(rng.random(3).astype(np.float32)).cuda()
        token = dw.sample_tokens(last, u, **setting)
        for r in range(3):
            s = dict(temperature=float(setting["temperature"][r]), top_k=int(setting["top_k"][r]), top_p=0.9)
            assert sr.accepted(last[r].double().cpu().numpy(), float(u[r]), int(token[r]), **s)
        text = [np.concatenate([t, [int(q)]]) for t, q in zip(text, token)]
        last = step(p, token, convs, states, slots)
        full = [prompt(p, dev(t), dev([0, len(t)]))[0][-1] for t in text]
        for r in range(3):
            assert (last[r] - full[r]).abs().max() <= 100 * D * 2.0 ** -24 * full[r].abs().max()
    assert (states[[1, 4]] == 0).all() and (convs[[1, 4]] == 0).all()


def train_pass(p, tokens, choice, dlogits):
    """Logits, and the gradients of table, convolution, rate, experts and head by hand; the router's choices are given."""
    b, l = tokens.shape
    e = dw.embedding_lookup(tokens, p["table"], scale=2.0)
    u = dw.causal_conv1d(e, p["w"], p["b"], activation="silu")
    gates = u @ p["gates"]
    h, saved = dw.gated_scan(u, gates[..., :D], gates[..., D:], p["rate"], save_for_grad=True)
    flat = h.view(-1, D)
    out, plan, weights, rows, y = experts(p, flat, choice)
    logits = out @ p["head"]
    dhead, dout = out.t() @ dlogits, dlogits @ p["head"].t()
    g = dw.expert_combine_grad(dout, y, plan, weights)
    drows, dexperts, ends = torch.zeros_like(rows), torch.zeros_like(p["experts"]), plan.offsets.tolist()
    for q in range(E):
        s = slice(ends[q], ends[q + 1])
        drows[s], dexperts[q] = g.dy[s] @ p["experts"][q].t(), rows[s].t() @ g.dy[s]
    score = flat @ p["router"]
    top = score.gather(1, score.topk(K, dim=1).indices)
    soft = torch.softmax(top, 1)
    dtop = soft * (g.dweights - (g.dweights * soft).sum(1, keepdim=True))
    dscore = torch.zeros_like(score).scatter_(1, score.topk(K, dim=1).indices, dtop)
    dh = dw.expert_dispatch_grad(drows, plan) + dscore @ p["router"].t()
    dgates = torch.empty_like(gates)
    s = dw.gated_scan_grad(dh.view_as(h), u, gates[..., :D], gates[..., D:], p["rate"], saved=saved, ddecay_gate=dgates[..., :D], dinput_gate=dgates[..., D:])
    du = s.dx + dgates @ p["gates"].t()
    c = dw.causal_conv1d_grad(du, e, p["w"], p["b"], activation="silu")
    dtable = dw.embedding_grad(tokens, c.dx, V, scale=2.0)
    return dict(logits=logits, head=dhead, experts=dexperts, rate=s.drate, w=c.dweight, b=c.dbias, table=dtable,
                gates=u.reshape(-1, D).t() @ dgates.view(-1, 2 * D))


def test_training_pass_matches_autograd_of_the_formulas():
    """Every gradient against torch.autograd in 64 bits on the host.  A gradient passes some 200 rows of the recurrence, sums
    over D channels and over all rows, each rounding 2^-24 of values that stay within 64 times its largest."""
    rng = np.random.default_rng(2)
    p = params(rng)
    b, l = 2, 90
    tokens = torch.from_numpy(rng.integers(-1, V, (b, l)).astype(np.int32)).cuda()
    choice = torch.from_numpy(np.stack([rng.permutation(E + 1)[:K] for _ in range(b * l)]).astype(np.int32)).cuda()  # E: no expert
    dlogits = randn(rng, b * l, V, scale=0.1)
    got = train_pass(p, tokens, choice, dlogits)
    leaf = {k: v.double().cpu().requires_grad_() for k, v in p.items()}
    tk, ch = tokens.cpu().long(), choice.cpu().long()
    e = torch.where((tk >= 0)[..., None], leaf["table"][tk.clamp(min=0)] * 2.0, 0.0)
    u = torch.nn.functional.silu(torch.nn.functional.pad(e, (0, 0, 3, 0)).unfold(1, 4, 1).mul(leaf["w"]).sum(-1) + leaf["b"])
    gates = torch.sigmoid(u @ leaf["gates"])
    a = torch.exp(leaf["rate"] * gates[..., :D])
    x = torch.sqrt(1 - a * a) * gates[..., D:] * u
    h, hs = torch.zeros(b, D, dtype=torch.float64), []
    for i in range(l):
        h = a[:, i] * h + x[:, i]
        hs.append(h)
    flat = torch.stack(hs, 1).view(-1, D)
    weights = torch.softmax((flat @ leaf["router"]).topk(K, dim=1).values, 1)
    out = 0
    for j in range(K):
        y = torch.bmm(flat[:, None], leaf["experts"][ch[:, j].clamp(max=E - 1)])[:, 0]
        out = out + torch.where((ch[:, j] < E)[:, None], weights[:, j:j + 1] * y, 0.0)
    logits = out @ leaf["head"]
    names = [k for k in got if k != "logits"]
    want = dict(zip(names, torch.autograd.grad(logits, [leaf[k] for k in names], dlogits.double().cpu())), logits=logits.detach())
    for k, g in got.items():
        assert g.shape == want[k].shape
        assert (g.double().cpu() - want[k]).abs().max() <= 2.0 ** -24 * 200 * 64 * want[k].abs().max(), k
