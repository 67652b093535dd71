"""The loss of sg_distill over the temperatures that it takes, against torch in 64
bits: at high ones the two distributions are nearly the same, and what is left of the
divergence counts T^2 times.

Tolerances (u = 2^-24; a = (max v - v) / T, d = (m - x) / T; c = log q - log p; C classes)
above T = 4, where the loss is T^2 (sum q (c + exp(-c) - 1) + rest), rest the entries'
lack of p: an exponential is off by (64 + 6 d) u, so q by Q = (80 + 6 a + 2 E[a]) u of
itself, p by P = (68 + 6 d + C / 256 + 2 E[d]) u, and log(z / z_q) by e = (140 + C / 256 + 8 E[d]
+ 8 E[a] + 2 |it|) u.  Each c has 4 (a + d) u of its own.  The first sum is off by its
terms times Q + 40 u, by |q - p| times c's own error, by rest e and by the square of both
together; where |c| is 1/2 and more, the term is q (c - 1) + p: 4 u (q |c| + q + p) and p P more.
The rest is off by its own p times P where the row is read again (below 1/8), by the
entries' p times P and 16 u otherwise; and the additions' leftovers by (C / 256)^2 u^2."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_distill import DT, INF, U, _case, _reference, _run, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _tolerance(x, ids, v, T):
    """(loss, its tolerance) of rows of which each class occurs once or more."""
    n, c = x.shape
    x, v, ids = x.double(), v.double(), ids.long()
    there = (ids >= 0) & (v > -INF)
    there = there & there[:, :1]
    at = ids.clamp(min=0)
    lowest = torch.full_like(v, -INF)
    top = torch.where(there, v, lowest).amax(1, keepdim=True)
    top = torch.where(top == -INF, torch.zeros_like(top), top)
    a = torch.where(there, (top - v) / T, torch.zeros_like(v))
    zq = torch.where(there, torch.exp(-a), torch.zeros_like(a)).sum(1, keepdim=True)
    zq = torch.where(zq == 0, torch.ones_like(zq), zq)
    q = torch.where(there, torch.exp(-a), torch.zeros_like(a)) / zq
    there = there & (q > 1e-36)  # (the others are 0, or nothing)
    d = (x.amax(1, keepdim=True) - x) / T
    z = torch.exp(-d).sum(1, keepdim=True)
    p = torch.exp(-d) / z
    zero = torch.zeros_like(a)
    pj, dj = torch.where(there, p.gather(1, at), zero), torch.where(there, d.gather(1, at), zero)
    apart = torch.log(z) - torch.log(zq)
    cj = torch.where(there, dj - a + apart, zero)
    near = torch.where(cj.abs() < 1e-4, cj * cj / 2 - cj ** 3 / 6, cj + torch.expm1(-cj))
    head = torch.where(there, q * near, zero).sum(1)
    # every class's p as often as it is no entry's
    counts = torch.zeros_like(p).scatter_add_(1, at, there.double())
    rest = (p * (1 - counts)).sum(1)
    loss = T * T * (head + rest)
    mean_d = torch.where(p > 0, p * d, torch.zeros_like(p)).sum(1, keepdim=True)
    mean_a = (q * a).sum(1, keepdim=True)
    P = torch.where(p > 0, p * (68 + 6 * d + c / 256 + 2 * mean_d) * U, torch.zeros_like(p))
    Pj = torch.where(there, P.gather(1, at), zero)
    e = ((140 + c / 256 + 8 * mean_d + 8 * mean_a + 2 * apart.abs()) * U)[:, 0]
    own = torch.where(there, 4 * (a + dj) * U, zero)
    tol = torch.where(there, q * near * (120 + 6 * a + 2 * mean_a) * U + (q - pj).abs() * own, zero).sum(1)
    tol += (p * (1 - counts).abs()).sum(1) * e + (e + own.amax(1)) ** 2
    far = there & (cj.abs() > 0.49)
    tol += torch.where(far, 4 * U * (q * cj.abs() + q + pj) + Pj, zero).sum(1)
    again, once = (P * (1 - counts).abs()).sum(1), Pj.sum(1) + 16 * U
    tol += torch.where(head + rest < 0.12, again, torch.where(head + rest > 0.13, once, torch.maximum(again, once)))
    tol += (c / 256 + 16) ** 2 * U * U
    none = ~((ids[:, 0] >= 0) & (v[:, 0] > -INF))
    return torch.where(none, torch.zeros_like(loss), loss), T * T * tol


def _hold(x, ids, v, T, mean=True, **kw):
    loss, total, grad = _run(x, ids, v, T, mean, **kw)
    want, tol = _tolerance(x, ids, v, T)
    off = (loss.double() - want).abs()
    assert bool((off <= tol).all()), (T, float((off / tol.clamp(min=1e-300)).max()), float((off / want.abs().clamp(min=1e-30)).max()))
    _, _, _, rows, g, gtol = _reference(x, ids, v, T, mean, 1.0)
    k = max(1, rows) if mean else 1
    assert float(total[1]) == rows
    assert abs(float(total[0]) - float(want.sum()) / k) <= (float(tol.sum()) + U * (len(x) / 1024 + 64) * float(want.abs().sum())) / k
    if grad is not None and grad.dtype == torch.float32:
        assert bool(((grad.double() - g).abs() <= gtol + 1e-44).all())
    return loss, total, grad


HOT = [4.0009765625, 6.0, 20.0, 100.0, 1000.0]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", [(1, 1, 1), (200, 128, 128), (40, 47, 47), (300, 47, 46), (2000, 100, 100), (33, 60, 128)])
@pytest.mark.parametrize("T", HOT)
def test_entries_of_all_classes(n, c, k, T, dt):
    x, ids, v = _case(n, c, k, dt, n + c)
    _hold(x, ids, v, T)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", [(20, 500, 20), (300, 1000, 64), (9, 2049, 33), (650, 2500, 128), (5, 16385, 5), (3, 50257, 64),
                                   (2, 131075, 128), (600, 9001, 30), (330, 50257, 20), (20001, 130, 2)])
@pytest.mark.parametrize("T", HOT)
def test_few_entries_of_many_classes(n, c, k, T, dt):
    x, ids, v = _case(n, c, k, dt, n + c + 1)
    _hold(x, ids, v, T)
    # nearly all of p with the entries: the others far below, in some rows not quite
    keep = torch.zeros((n, c), dtype=torch.bool, device="cuda").scatter_(1, ids.long().clamp(min=0), True)
    level = torch.tensor([8.0, 14.0, 20.0, 60.0], device="cuda").repeat((n + 3) // 4)[:n, None] * T
    x = torch.where(keep, x.float(), x.float() - level).to(DT[dt])
    first = _hold(x, ids, v, T)
    again = _run(x, ids, v, T)
    assert all(torch.equal(s, t) for s, t in zip(first, again))  # the same bits
    only = _run(x, ids, v, T, grad=False)
    assert torch.equal(only[0], first[0]) and torch.equal(only[1], first[1])
    alone = _run(x, ids, v, T, total=False)
    assert torch.equal(alone[0], first[0])


@pytest.mark.parametrize("n,c", [(50, 96), (6, 3000), (700, 2500), (3, 50257), (170, 50257)])
@pytest.mark.parametrize("T", HOT)
@pytest.mark.parametrize("noise", [0.0, 1e-3, 0.1])
def test_a_student_close_to_its_teacher(n, c, T, noise):
    k = min(c, 128)
    x, ids, v = _case(n, c, k, "f32", c)
    ids = ids.clamp(min=0) if k < 3 else ids
    g = torch.Generator("cuda").manual_seed(c)
    keep = torch.zeros((n, c), dtype=torch.bool, device="cuda").scatter_(1, ids.long().clamp(min=0), True)
    x = torch.where(keep, x, torch.full_like(x, -INF))
    x.scatter_(1, ids.long().clamp(min=0), v.clamp(min=-10) - 7 + noise * torch.randn(v.shape, generator=g, device="cuda"))
    x = torch.where(torch.isinf(x) & (ids[:, :1] < 0), torch.zeros_like(x), x)
    v = v.clamp(min=-10)
    _hold(x, ids, v, T)


@pytest.mark.parametrize("n,c,k", [(40, 60, 12), (20, 900, 64), (6, 40001, 40), (400, 9001, 16)])
@pytest.mark.parametrize("T", [5.0, 300.0])
def test_classes_that_occur_more_than_once(n, c, k, T):
    x, ids, v = _case(n, c, k, "f32", c)
    ids = ids.clamp(min=0)
    ids[:, k // 3:] = ids[:, k // 3:k // 3 + 1]
    v = torch.nan_to_num(v, neginf=0.0)
    _hold(x, ids, v, T)
    _hold(x.masked_fill_(torch.zeros_like(x, dtype=torch.bool).scatter_(1, ids.long(), True).logical_not_(), -INF), ids, v, T)


@pytest.mark.parametrize("n,c", [(37, 47), (200, 128), (37, 5001), (700, 2500), (500, 9001)])
def test_rows_behind_the_count_and_no_rows(n, c):
    x, ids, v = _case(n, c, 9, "f32", c)
    T, m = 50.0, n * 3 // 5
    for count in (m, 0, n + 3):
        loss, total, grad = torch.full((n,), 7.0, device="cuda"), torch.full((2,), 7.0, device="cuda"), torch.full_like(x, 7.0)
        need = sg.sg_distill_workspace(n, c)
        ws = sg.aligned_workspace(need + 4096)
        ws.fill_(0xCD)
        sg.sg_distill(x, ids, v, n, torch.tensor([count], dtype=torch.int32, device="cuda"), loss, total, grad, ws[:need], temperature=T)
        sg.sg_stream_check()
        r = min(count, n)
        want, tol = _tolerance(x[:r], ids[:r], v[:r], T) if r else (torch.zeros(0), torch.zeros(0))
        assert bool(((loss[:r].double() - want.to(loss.device)).abs() <= tol.to(loss.device)).all())
        assert bool((loss[r:] == 7).all()) and bool((grad[r:] == 7).all()) and bool((ws[need:] == 0xCD).all())
        used = int(((ids[:r, 0] >= 0) & (v[:r, 0] > -INF)).sum())
        assert float(total[1]) == used and (r > 0 or float(total[0]) == 0)
    e = torch.empty(0, device="cuda")
    total = torch.full((2,), 7.0, device="cuda")
    sg.sg_distill(x[:0], ids[:0], v[:0], 0, None, e, total, None, _ws(0, c), temperature=T)
    sg.sg_stream_check()
    assert bool((total == 0).all())


@pytest.mark.parametrize("n,c", [(30, 100), (30, 900), (6, 40000), (700, 9000), (700, 2500)])
def test_bad_values_and_masked_classes(n, c):
    x, ids, v = _case(n, c, 6, "f32", c)
    clean = _run(x, ids, v, 30.0, mean=False)
    hit = torch.arange(n, device="cuda") % 3 == 0
    hit &= (ids[:, 0] >= 0) & (v[:, 0] > -INF)
    for bad in (float("nan"), INF):
        y = x.clone()
        y[hit, c // 2] = bad
        got = _run(y, ids, v, 30.0, mean=False)
        assert bool(torch.isnan(got[0][hit]).all()) and torch.equal(got[0][~hit], clean[0][~hit])
        w = v.clone()
        w[hit, 0] = bad
        got = _run(x, ids, w, 30.0, mean=False)
        assert bool(torch.isnan(got[0][hit]).all()) and torch.equal(got[0][~hit], clean[0][~hit])
    y = x.clone()
    y[0] = -INF
    y[4, ids[4, 0].long()] = -INF  # a class that has q
    got = _run(y, ids, v, 30.0, mean=False)
    assert float(got[0][0]) == INF and float(got[0][4]) == INF and float(got[1][0]) == INF
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[0] = keep[4] = False
    assert torch.equal(got[0][keep], clean[0][keep])
    assert not np.isnan(float(got[1][0]))


def test_graphs_and_streams_with_hot_losses():
    cases = [_case(64, 100, 8, "f32", 1), _case(6, 40001, 40, "f32", 2), _case(700, 2500, 5, "bf16", 3), _case(700, 9001, 8, "bf16", 4)]
    want = [_run(*t, 20.0) for t in cases]
    shared = _ws(700, 40001)
    outs = [[torch.empty_like(t) for t in w] for w in want]
    graphs = []
    torch.cuda.synchronize()
    for t, o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sg.sg_distill(*t, len(t[0]), None, *o, shared, temperature=20.0)
        graphs.append(graph)
    for graph in graphs + graphs[::-1]:
        graph.replay()
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(s, t) for w, o in zip(want, outs) for s, t in zip(w, o))
    for o in outs:
        for t in o:
            t.fill_(7.0)
    ws = [_ws(*t[0].shape) for t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, o, s, m in zip(cases, outs, streams, ws):
            sg.sg_distill(*t, len(t[0]), None, *o, m, temperature=20.0, stream=s)
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(s, t) for w, o in zip(want, outs) for s, t in zip(w, o))
