"""The experts' moves under plans that leave rows out: room between the experts, choices dropped after the split.  New
tensors are zero there, whatever the memory held before."""
import ctypes

import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
from device_wide_prefix_tile_amd import experts, sequence as seq

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def leave_nan(shape, t):
    """The next tensor of that size is made of memory that holds NaN."""
    torch.cuda.synchronize()
    q = torch.full(shape, float("nan"), dtype=t, device="cuda")
    torch.cuda.synchronize()
    del q


def expected(x, places, rows):
    """out[places[t, j]] = x[t] on the host, zero elsewhere; the last choice wins (places do not repeat here)."""
    out = torch.zeros(rows, x.shape[1], dtype=x.dtype)
    p, src = places.cpu(), x.cpu()
    for j in range(p.shape[1]):
        ok = (p[:, j] >= 0) & (p[:, j] < rows)
        out[p[ok, j].long()] = src[ok]
    return out


def check(x, plan, rows, what):
    n, k = plan.places.shape
    d = x.shape[1]
    leave_nan((n * k, d), x.dtype)
    got = dw.expert_dispatch(x, plan)
    assert torch.equal(got.cpu(), expected(x, plan.places, n * k)), "%s: dispatch" % what
    y = torch.ones(rows, d, dtype=x.dtype, device="cuda")
    for w in (torch.ones(n, k, device="cuda"), None):
        leave_nan((rows, d), x.dtype)
        g = dw.expert_combine_grad(x, y, plan, w)
        assert torch.equal(g.dy.cpu(), expected(x, plan.places, rows)), "%s: gradient" % what


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("n,k,e,d", [(1, 1, 1, 8), (40, 2, 8, 64), (33, 5, 7, 515), (700, 8, 32, 136), (3000, 4, 16, 590)])
def test_choices_dropped_after_the_split(t, n, k, e, d):
    """A capacity for every expert: choices beyond it lose their place, rows below the number of rows with an expert stay empty."""
    rng = np.random.default_rng(n + d)
    x = torch.from_numpy(rng.standard_normal((n, d))).to(T[t]).cuda()
    plan = dw.expert_split(torch.from_numpy(rng.integers(-1, e, (n, k)).astype(np.int32)).cuda(), e)
    for capacity in (0, 1, max(1, n * k // e // 2)):
        o = plan.offsets.long()
        expert = torch.searchsorted(o[1:], plan.places.clamp(min=0).long(), right=True).clamp(max=e - 1)
        over = plan.places - plan.offsets[expert] >= capacity
        dropped = plan._replace(places=torch.where(over, -1, plan.places).contiguous())
        check(x, dropped, n * k, "capacity %d" % capacity)
        check(x, dropped, n * k + 70, "capacity %d, more rows" % capacity)
    kept = plan.places.clone()
    plan.places[::2] = -1  # in place
    check(x, plan, n * k, "every other token")
    plan.places.copy_(kept)
    check(x, plan, n * k, "all of them again")


@pytest.mark.parametrize("t", list(T))
def test_room_between_the_experts(t):
    """Places of a plan that was made elsewhere: each expert's rows start at a multiple of 64; offsets say nothing of use."""
    rng = np.random.default_rng(3)
    n, k, e, d, room = 200, 2, 5, 72, 64
    c = rng.integers(0, e, (n, k))
    places, rows = np.full((n, k), -1), 0
    for q in range(e):
        at = np.argwhere(c == q)
        for i, (a, j) in enumerate(at):
            places[a, j] = rows + i
        rows += (len(at) + room - 1) // room * room
    x = torch.from_numpy(rng.standard_normal((n, d))).to(T[t]).cuda()
    places = torch.from_numpy(places.astype(np.int32)).cuda()
    for ends in ([0, rows], [0, 3], [7, 2 ** 31 - 1], [0, -9]):
        plan = dw.ExpertPlan(torch.tensor(ends, dtype=torch.int32, device="cuda"), places, torch.zeros(0, dtype=torch.int32, device="cuda"))
        check(x, plan, rows, "room")


def test_many_rows_of_no_choice():
    """More rows than are looked at at a time, places in some of them; rows of 2^32 bytes and more."""
    rng = np.random.default_rng(4)
    rows, d, n, k = 40_000_000, 64, 50, 4
    x = torch.from_numpy(rng.standard_normal((n, d))).to(torch.bfloat16).cuda()
    at = np.unique(np.concatenate([rng.integers(0, rows, n * k - 4), [0, rows - 1, 65535, 65536]]))
    places = np.full(n * k, -1)
    places[rng.permutation(n * k)[:at.size]] = at
    places = torch.from_numpy(places.astype(np.int32)).view(n, k).cuda()
    plan = dw.ExpertPlan(torch.zeros(2, dtype=torch.int32, device="cuda"), places, places.view(-1))
    y = torch.ones(rows, d, dtype=torch.bfloat16, device="cuda")
    leave_nan((rows, d), torch.bfloat16)
    g = dw.expert_combine_grad(x, y, plan)
    live = places.view(-1) >= 0
    to = places.view(-1)[live].long()
    assert torch.equal(g.dy[to], x[torch.nonzero(live)[:, 0] // k])
    g.dy[to] = 0
    assert int(torch.count_nonzero(g.dy)) == 0 and not g.dy.isnan().any()


def guarded(rows, d, guard=9):
    whole = torch.full((rows + 2 * guard, d), 5.0, device="cuda")
    return whole, whole[guard:guard + rows]


@pytest.mark.parametrize("end", [-5, -2 ** 31, 0, 3, 11, 12, 13, 2 ** 31 - 1])
def test_rows_used_through_the_c_entry(end):
    """`used` of any value: rows from there on that no place leads to become zero, others and everything outside the array
    are left as they were."""
    rng = np.random.default_rng(5)
    n, k, d, rows = 4, 2, 40, 12
    x = torch.from_numpy(rng.standard_normal((n, d))).float().cuda()
    places = torch.tensor([[0, 9], [3, -1], [5, 100], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    used = torch.tensor([end], dtype=torch.int32, device="cuda")
    want = torch.full((rows, d), 5.0)
    want[max(0, min(end, rows)):] = 0
    for r, t in ((0, 0), (9, 0), (3, 1), (5, 2)):
        want[r] = x[t].cpu()
    whole, out = guarded(rows, d)
    handle = torch.cuda.current_stream().cuda_stream
    a = experts._DispatchArgs(dtype=0, tokens=n, rows=rows, choices=k, channels=d, places=places.data_ptr(), used=used.data_ptr(), x=x.data_ptr(),
                              x_stride=d, out=out.data_ptr(), out_stride=d)
    assert seq._lib().expert_dispatch(ctypes.byref(a), handle) == 0
    assert torch.equal(out.cpu(), want) and (whole[:9] == 5.0).all() and (whole[9 + rows:] == 5.0).all()
    whole, out = guarded(rows, d)
    a = experts._CombineGradArgs(dtype=0, tokens=n, rows=rows, choices=k, channels=d, places=places.data_ptr(), used=used.data_ptr(),
                                 dout=x.data_ptr(), dout_stride=d, dy=out.data_ptr(), dy_stride=d)
    assert seq._lib().expert_combine_grad(ctypes.byref(a), handle) == 0
    assert torch.equal(out.cpu(), want) and (whole[:9] == 5.0).all() and (whole[9 + rows:] == 5.0).all()


def test_graphs_with_dropped_choices():
    """Captured with one plan, replayed with the places of another."""
    rng = np.random.default_rng(6)
    n, k, e, d = 500, 4, 16, 96
    x = torch.from_numpy(rng.standard_normal((n, d))).float().cuda()
    plan = dw.expert_split(torch.from_numpy(rng.integers(0, e, (n, k)).astype(np.int32)).cuda(), e)
    y, all_places = torch.ones(n * k, d, device="cuda"), plan.places.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            rows, grad = dw.expert_dispatch(x, plan), dw.expert_combine_grad(x, y, plan)
    for step in (1, 2, 3, 5):
        plan.places.copy_(all_places)
        plan.places[::step] = -1
        rows.fill_(float("nan"))
        grad.dy.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = expected(x, plan.places, n * k)
        assert torch.equal(rows.cpu(), want) and torch.equal(grad.dy.cpu(), want)
