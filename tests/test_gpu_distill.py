"""Distillation from a teacher's top logits (sg_distill) against torch in 64
bits.

Tolerances (u = 2^-24; d = (m - x) / T, m the row's maximum): an exponential's
argument is rounded three times (the difference, log2(e) / T, the product) and the
base-2 exponential is off by 2^-22, so p is off by p (64 + 6 d + C / 256 + 2 E[d]) u
with its sum, and q by q (80 + 6 a + 2 E[a]) u likewise, a = (max v - v) / T.  The gradient is off by w T times both, plus
4 u of the larger part; the loss by T^2 times sum q (|log q - log p| (80 + 6 a + 2 E[a])
+ 4 (a + d + log z_q + log z) + 160 + C / 256 + 2 E[d]) u.  A bf16 gradient has to be the
rounding of a value within that."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_xent_rows import _rounded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _ws(n, c):
    ws = sg.aligned_workspace(sg.sg_distill_workspace(n, c))
    ws.fill_(0xCD)
    return ws


def _run(x, ids, v, T, mean=True, gs=1.0, grad=True, d_n=None, total=True, reported=False):
    n, c = x.shape
    loss, tot = torch.full((n,), 7.0, device="cuda"), torch.full((2,), 7.0, device="cuda") if total else None
    g = torch.full((n, c), 7.0, device="cuda", dtype=x.dtype) if grad else None
    sg.sg_distill(x, ids, v, n, d_n, loss, tot, g, _ws(n, c), temperature=T, mean=mean, grad_scale=gs)
    if reported:  # classes out of range
        with pytest.raises(sg.SgError) as e:
            sg.sg_stream_check()
        assert e.value.status == sg.SG_ERR_INVALID_INDEX
    else:
        sg.sg_stream_check()
    return loss, tot, g


def _reference(x, ids, v, T, mean, gs):
    """(loss, its tolerance, total, rows, gradient, its tolerance)."""
    n, c = x.shape
    x, v, ids = x.double(), v.double(), ids.long()
    there = (ids >= 0) & (v > -INF)
    used = there[:, 0]
    there = there & used[:, None]
    a = torch.where(there, v, -INF)
    top = torch.where(used, a.amax(1), torch.zeros_like(a[:, 0]))[:, None]
    a = torch.where(there, (top - v) / T, torch.zeros_like(v))
    e = torch.where(there, torch.exp(-a), torch.zeros_like(v))
    zq = torch.where(used, e.sum(1), torch.ones_like(top[:, 0]))[:, None]
    q = e / zq
    m = x.amax(1, keepdim=True)
    none = m == -INF
    m = torch.where(none, torch.zeros_like(m), m)
    d = (m - x) / T
    ex = torch.exp(-d)
    z = ex.sum(1, keepdim=True)
    p = ex / z.clamp(min=1e-300)
    mean_d = torch.where(p > 0, p * d, torch.zeros_like(d)).sum(1, keepdim=True)
    mean_a = (q * a).sum(1, keepdim=True)
    at = ids.clamp(min=0)
    dj = torch.where(there, d.gather(1, at), torch.zeros_like(a))
    log_z, log_zq = torch.log(torch.where(none, torch.ones_like(z), z)), torch.log(zq)  # (nothing left: dj is inf)
    term = (-a - log_zq) + (log_z + dj)
    term = torch.where(q > 0, term, torch.zeros_like(term))
    loss = T * T * torch.where(q > 0, q * term, torch.zeros_like(q)).sum(1)
    big = (term.abs() * (80 + 6 * a + 2 * mean_a) + 4 * (a + dj + log_zq + log_z) + 160 + c / 256 + 2 * mean_d)
    ltol = T * T * U * torch.where(q > 0, q * big, torch.zeros_like(q)).sum(1)
    rows = int(used.sum())
    w = gs / max(1, rows) if mean else gs
    scale = (w * T * used * ~none[:, 0])[:, None]
    grad = (p.clone().scatter_add_(1, at, -q)) * scale
    tol = torch.where(p > 0, p * (68 + 6 * d + c / 256 + 2 * mean_d), torch.zeros_like(p))
    tol.scatter_add_(1, at, q * (84 + 6 * a + 2 * mean_a))
    total = loss.sum() / (max(1, rows) if mean else 1)
    return loss, ltol, total, rows, grad, tol * scale.abs() * U


def _hold(x, ids, v, T, mean, gs, got):
    loss, total, grad = got
    want, ltol, tot, rows, g, tol = _reference(x, ids, v, T, mean, gs)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isposinf(loss.double()), torch.isposinf(want))
    off = (loss.double() - want).abs()
    assert bool((off <= ltol)[fin].all()), float((off / ltol)[fin].max())
    if total is not None:
        assert float(total[1]) == rows
        if bool(fin.all()):
            k = max(1, rows) if mean else 1
            assert abs(float(total[0]) - float(tot)) <= float(ltol.sum()) / k + U * (len(x) / 1024 + 64) * float(
                want.abs().sum()) / k
        else:
            assert float(total[0]) == INF
    if grad is None:
        return
    if grad.dtype == torch.bfloat16:
        assert bool(((_rounded(g - tol - 1e-40) <= grad.double()) & (grad.double() <= _rounded(g + tol + 1e-40))).all())
    else:
        bad = (grad.double() - g).abs() - tol
        assert bool((bad <= 1e-44).all()), float(bad.max())


def _case(n, c, k, dt, seed, spread=2.0):
    """Logits, k distinct classes of each row in any order, values; some rows have
    fewer entries, some none."""
    g = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    k = min(k, c)
    ids = torch.stack([torch.from_numpy(rng.permutation(c)[:k] if c < 5000 else rng.choice(c, k, replace=False)) for _ in range(n)])
    ids = ids.to(torch.int32).cuda()
    v = 3 * torch.randn((n, k), generator=g, device="cuda") + 5
    x = spread * torch.randn((n, c), generator=g, device="cuda")
    x.scatter_add_(1, ids.long(), 0.7 * v)
    if n > 3:
        ids[2] = -1
        ids[1, k // 2 + 1:] = -1
        v[3, 1:] = -INF
    if n > 8:
        v[5, 0] = -INF  # no teacher
        ids[7, 0] = -1  # no teacher, whatever follows
    return x.to(DT[dt]), ids, v


SIZES = [(1, 1, 1), (1, 2, 2), (5, 31, 8), (256, 128, 8), (300, 47, 47), (129, 127, 128), (33, 500, 20), (17, 1025, 100),
         (40, 1000, 64), (3001, 40, 5), (9, 2049, 33), (7, 8191, 64), (5, 16385, 5), (3, 50257, 64), (4, 131072, 64),
         (2, 131075, 128), (1, 300001, 20), (1200, 2500, 20), (600, 9001, 30), (330, 50257, 20), (200, 100001, 128),
         (170, 150001, 10), (20001, 130, 2), (40, 600, 128)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", SIZES)
def test_loss_and_gradient(n, c, k, dt):
    x, ids, v = _case(n, c, k, dt, n * 7 + c)
    for T, mean, gs in ((2.0, True, 1.0), (0.7, False, -0.25)):
        got = _run(x, ids, v, T, mean, gs)
        _hold(x, ids, v, T, mean, gs, got)
    again = _run(x, ids, v, T, mean, gs)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits
    only = _run(x, ids, v, T, mean, gs, grad=False)
    assert torch.equal(only[0], got[0]) and torch.equal(only[1], got[1])
    part = _run(x, ids, v, T, mean, gs, total=False)
    assert torch.equal(part[0], got[0]) and torch.equal(part[2], got[2])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vecs", [256, 257, 384, 385, 512, 513])
@pytest.mark.parametrize("k", [1, 32, 33, 128])
def test_many_rows_at_the_ends_of_the_forms(vecs, k, dt):
    # a warp a row in 8, 12 or 16 vectors a lane, blocks from there on
    n, c = 701, vecs * (4 if dt == "f32" else 8)
    x, ids, v = _case(n, c, k, dt, vecs + k)
    if k > 2:
        ids[11, 2:] = ids[11, 1:2]  # one class many times
        ids[12, 1] = ids[12, 0]
    x[13], x[14, c // 2:] = -INF, -INF
    _hold(x, ids, v, 2.0, True, 1.0, _run(x, ids, v, 2.0))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", [(40, 60, 12), (20, 900, 64), (9, 3000, 100), (6, 40001, 40), (400, 9001, 16), (1300, 2500, 8)])
def test_classes_that_occur_more_than_once(n, c, k, dt):
    x, ids, v = _case(n, c, k, dt, c)
    ids[:, k // 3:] = ids[:, k // 3:k // 3 + 1]                        # one class many times
    ids[::2, : k // 3] = ids[::2, : k // 3] // (c // 4 + 1) * (c // 4)  # a few of each
    ids[9 % n] = c - 1
    wrong = bool((ids < -1).any())  # (row 2 had none: its first entries are out of range now)
    for T in (1.0, 4.0):
        _hold(x, ids, v, T, True, 1.0, _run(x, ids, v, T, reported=wrong))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", [(40, 60, 12), (20, 900, 64), (6, 40001, 40), (400, 9001, 16)])
@pytest.mark.parametrize("mask", [-INF, -1e9, "lowest"])
def test_masked_classes(n, c, k, mask, dt):
    x, ids, v = _case(n, c, k, dt, c + 1)
    value = torch.finfo(DT[dt]).min if mask == "lowest" else mask
    off = torch.rand((n, c), generator=torch.Generator("cuda").manual_seed(k), device="cuda") < 0.5
    keep = torch.zeros((n, c), dtype=torch.bool, device="cuda").scatter_(1, ids.long().clamp(min=0), True)
    x = torch.where(off & ~keep, torch.full_like(x, value), x)
    _hold(x, ids, v, 2.0, True, 1.0, _run(x, ids, v, 2.0))
    if mask != -INF:
        return
    x[0] = -INF               # nothing left
    x[1, ids[1, 0].long()] = -INF  # the teacher's own class
    _hold(x, ids, v, 2.0, True, 1.0, _run(x, ids, v, 2.0))


@pytest.mark.parametrize("c", [40, 1500, 9001])
def test_levels(c):
    # neither the logits' nor the values' level counts
    levels = [0.0, 1e3, -1e3, 1e5, -1e6, 1e9, -1e20, 3e38]
    x, ids, v = _case(8, c, 6, "f32", c)
    ids = ids.clamp(min=0)
    for s in range(8):
        x[s] = torch.full((c,), levels[s], device="cuda") if abs(levels[s]) > 1e6 else x[s] + levels[s]
        v[s] = torch.nan_to_num(v[s], neginf=0.0) if abs(levels[s]) <= 1e6 else 1.0
        v[s] += levels[(s + 3) % 8] if abs(levels[(s + 3) % 8]) < 1e6 else 0
    _hold(x, ids, v, 2.0, True, 1.0, _run(x, ids, v, 2.0))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", [(30, 100), (30, 900), (6, 40000), (700, 9000)])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_nan_and_inf_stay_in_their_row(n, c, bad, dt):
    x, ids, v = _case(n, c, 6, dt, c)
    clean = _run(x, ids, v, 2.0, mean=False)
    hit = torch.arange(n, device="cuda") % 3 == 0
    hit &= (ids[:, 0] >= 0) & (v[:, 0] > -INF)
    y = x.clone()
    y[hit, c // 2] = bad
    got = _run(y, ids, v, 2.0, mean=False)
    assert bool(torch.isnan(got[0][hit]).all()) and bool(torch.isnan(got[2][hit]).all())
    assert torch.equal(got[0][~hit], clean[0][~hit]) and torch.equal(got[2][~hit], clean[2][~hit])
    w = v.clone()
    w[hit, 0] = bad
    got = _run(x, ids, w, 2.0, mean=False)
    at = torch.where(ids >= 0, ids, ids[:, :1]).long()
    assert bool(torch.isnan(got[0][hit]).all()) and bool(torch.isnan(got[2].gather(1, at.clamp(min=0))[hit, 0]).all())
    assert torch.equal(got[0][~hit], clean[0][~hit]) and torch.equal(got[2][~hit], clean[2][~hit])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", [(37, 47), (37, 1001), (37, 5001), (500, 9001), (5, 70000)])
@pytest.mark.parametrize("start,gap", [(1, 3), (3, 8), (0, 1)])
def test_strides_and_rows_behind_the_count(n, c, start, gap, dt):
    x, ids, v = _case(n, c, 9, dt, c)
    k, m = ids.shape[1], n * 3 // 5
    wide = torch.full((n, start + c + gap), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, start:start + c] = x
    out = torch.full((n, 2 + c + 2 * gap), 7.0, dtype=x.dtype, device="cuda")
    for count in (m, 0, n + 3):
        out.fill_(7.0)
        loss, total = torch.full((n,), 7.0, device="cuda"), torch.full((2,), 7.0, device="cuda")
        sg.sg_distill(wide[:, start:start + c], ids, v, n, torch.tensor([count], dtype=torch.int32, device="cuda"), loss, total,
                      out[:, 2:2 + c], _ws(n, c), temperature=2.0)
        sg.sg_stream_check()
        r = min(count, n)
        _hold(x[:r], ids[:r], v[:r], 2.0, True, 1.0, (loss[:r], total, out[:r, 2:2 + c]))
        assert bool((loss[r:] == 7).all()) and bool((out[r:] == 7).all())
        assert bool((out[:, :2] == 7).all()) and bool((out[:, 2 + c:] == 7).all())


def test_gradient_is_the_losss_slope():
    # central differences of the loss in 64 bits; the second derivative of the loss is
    # at most 1 in each logit, the third 1, so a step of 1e-4 leaves 1e-8 / 6
    x, ids, v = _case(4, 23, 5, "f32", 3)
    ids[0, 3] = ids[0, 1]
    T, h = 2.0, 1e-4
    grad = _run(x, ids, v, T, mean=False)[2].double()

    def loss_at(y):
        return _reference(y, ids, v, T, False, 1.0)[0]
    for c in range(23):
        step = torch.zeros(23, dtype=torch.float64, device="cuda")
        step[c] = h
        slope = (loss_at(x.double() + step) - loss_at(x.double() - step)) / (2 * h)
        assert float((slope - grad[:, c]).abs().max()) <= 1e-6


def test_classes_out_of_range_are_reported():
    for n, c in ((9, 40), (9, 5000), (700, 9001)):
        x, ids, v = _case(n, c, 5, "f32", 1)
        ids[0, 2], ids[4, 0] = c, -2
        loss, total, grad = torch.empty(n, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
        sg.sg_distill(x, ids, v, n, None, loss, total, grad, _ws(n, c), temperature=1.0)
        with pytest.raises(sg.SgError) as e:
            sg.sg_stream_check()
        assert e.value.status == sg.SG_ERR_INVALID_INDEX
        ids[0, 2] = ids[4, 0] = -1
        want = _run(x, ids, v, 1.0)
        assert all(torch.equal(a, b) for a, b in zip((loss, total, grad), want))


def test_offsets_past_32_bits():
    n, c = 33000, 70001
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty((n, c), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = torch.randint(0, c, (n, 3), generator=g, device="cuda", dtype=torch.int32)
    v = torch.randn((n, 3), generator=g, device="cuda")
    loss, total, grad = _run(x, ids, v, 1.0, mean=False)
    at = torch.tensor([0, 1, 17000, 30678, 30679, n - 1], device="cuda")
    _hold(x[at], ids[at], v[at], 1.0, False, 1.0, (loss[at], None, grad[at]))


def test_two_graphs_share_a_workspace():
    cases = [_case(64, c, 8, "f32", c) for c in (100, 5000)] + [_case(700, 9001, 8, "bf16", 1)]
    want = [_run(*t, 2.0) for t in cases]
    ws = _ws(700, 9001)
    outs = [[torch.empty_like(t) for t in w] for w in want]
    graphs = []
    torch.cuda.synchronize()
    for t, o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sg.sg_distill(*t, len(t[0]), None, *o, ws, temperature=2.0)
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs + graphs[::-1]:
            graph.replay()
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))


def test_two_streams_at_once():
    # long rows streamed, few long rows, a small call in one cluster, a row a warp
    cases = [_case(700, 9001, 8, "bf16", 1), _case(9, 40001, 40, "f32", 2), _case(200, 100, 8, "f32", 3), _case(2000, 2500, 5, "f32", 4)]
    want = [_run(*t, 2.0) for t in cases]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    ws = [_ws(*t[0].shape) for t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, o, s, m in zip(cases, outs, streams, ws):
            sg.sg_distill(*t, len(t[0]), None, *o, m, temperature=2.0, stream=s)
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("start,gap", [(1, 3), (3, 8), (0, 1), (0, 0)])
def test_many_rows_at_any_alignment(start, gap, dt):
    n, c = 650, 1801 if dt == "f32" else 3601
    x, ids, v = _case(n, c, 9, dt, start)
    wide = torch.full((n, start + c + gap), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, start:start + c] = x
    out = torch.full((n, 2 + c + gap), 7.0, dtype=x.dtype, device="cuda")
    loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    m = n - 13
    sg.sg_distill(wide[:, start:start + c], ids, v, n, torch.tensor([m], dtype=torch.int32, device="cuda"), loss, total,
                  out[:, 2:2 + c], _ws(n, c), temperature=2.0)
    sg.sg_stream_check()
    _hold(x[:m], ids[:m], v[:m], 2.0, True, 1.0, (loss[:m], total, out[:m, 2:2 + c]))
    out[:m, 2:2 + c] = 7.0
    assert bool((out == 7).all())


def test_answers_of_a_teacher_train_a_student():
    # a teacher's top logits as sg_logprobs reports them, then the student's loss and
    # gradient: with every class reported, the full divergence and its gradient
    g = torch.Generator("cuda").manual_seed(2)
    n, c, T = 50, 96, 2.0
    teacher, student = (2 * torch.randn((n, c), generator=g, device="cuda") for _ in range(2))
    ids, lps = torch.empty((n, c), dtype=torch.int32, device="cuda"), torch.empty((n, c), device="cuda")
    sg.sg_logprobs(teacher, None, n, None, None, None, ids, lps)
    loss, total, grad = _run(student, ids, lps, T)
    s = student.double().requires_grad_()
    want = torch.nn.functional.kl_div(torch.log_softmax(s / T, 1), torch.softmax(teacher.double() / T, 1),
                                      reduction="batchmean") * T * T
    want.backward()
    # (values rounded to fp32: 2^-24 of about 8; p and q as above with d, a below 10)
    assert abs(float(total[0]) - float(want.detach())) <= 300 * U * (1 + float(want.detach()))
    assert float((grad.double() - s.grad).abs().max()) <= T / n * 200 * U
