"""Softmax cross-entropy with gradient (sg_xent) against plain numpy in 64
bits.

Tolerances (u = 2^-24): an exponential of an fp32 argument d <= 0 is off by
(8 + 2 |d|) u relative (two roundings of the argument and the hardware
base-2 exponential's 2^-22), the sum of C terms by (C / 256 + 32) u, so a
probability by e = (64 + 4 |d| + C / 256) u relative with the error of the sum
(a mean of such errors, whose mean |d| stays below 16 here); the gradient by
w (p e + 2 u), the loss by u (|max| + |x_label| + |log z|) 4 plus the sum's
error (128 + C / 256) u.  A bf16 gradient has to be the rounding of a value
within that tolerance."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from rounding import within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _reference(x, labels, mean, gs):
    n, c = x.shape
    valid = int((labels != -1).sum())
    w = gs / max(1, valid) if mean else gs
    loss, grad, err = np.zeros(n), np.zeros((n, c)), np.zeros((n, c))
    lerr = np.zeros(n)
    for r in range(n):
        y = labels[r]
        if y == -1:
            continue
        m = x[r].max()
        if m == -np.inf:
            loss[r] = np.inf
            continue
        with np.errstate(invalid="ignore"):
            e = np.exp(x[r] - m)
        z = e.sum()
        p = e / z
        d = np.where(np.isfinite(x[r]), m - x[r], 0.0)
        loss[r] = np.log(z) + (m - x[r, y])
        grad[r] = w * p
        grad[r, y] -= w
        err[r] = abs(w) * (p * (64 + 4 * d + c / 256) + 2) * U
        xy = abs(x[r, y]) if np.isfinite(x[r, y]) else 0.0
        lerr[r] = U * (4 * (abs(m) + xy + abs(np.log(z))) + 128 + c / 256)
    total = loss.sum() / max(1, valid) if mean else loss.sum()
    return loss, lerr, total, valid, grad, err


def _logits(rng, n, c, dt, spread=2.0):
    return torch.from_numpy((spread * rng.standard_normal((n, c))).astype(np.float32)).cuda().to(DT[dt])


def _check(x, labels, loss, total, grad, mean, gs, n=None):
    n = x.shape[0] if n is None else n
    lo, lerr, tot, valid, gr, err = _reference(x[:n].double().cpu().numpy(), labels[:n], mean, gs)
    got = loss[:n].double().cpu().numpy()
    fin = np.isfinite(lo)
    assert np.array_equal(np.isposinf(got), np.isposinf(lo))
    assert np.all(np.abs(got[fin] - lo[fin]) <= lerr[fin])
    if total is not None:
        t = total.double().cpu().numpy()
        assert t[1] == valid
        if fin.all():
            k = max(1, valid) if mean else 1
            assert abs(t[0] - tot) <= (lerr.sum() + (len(lo) / 1024 + 48) * U * np.abs(lo).sum()) / k + U * abs(tot)
        else:
            assert np.isposinf(t[0])
    if grad is not None:
        g = grad[:n].double().cpu().numpy()
        assert np.all(within(g, gr, err + 2.0 ** -148, grad.dtype == torch.bfloat16))


def _ws(n, c):
    ws = sg.aligned_workspace(sg.sg_xent_workspace(n, c))
    ws.fill_(0xCD)
    return ws


@pytest.mark.parametrize("n,c", [(1, 1), (1, 2), (3, 31), (5, 32), (256, 128), (300, 172), (129, 127), (40, 1000),
                                 (17, 1025), (9, 4096), (7, 8191), (5, 8193), (4, 16385), (3, 32771), (3, 50257),
                                 (2, 65536), (1, 131072), (2, 131075), (1, 300001), (5000, 7), (4097, 40),
                                 (30001, 16), (20000, 17), (70000, 3), (9000, 130), (3000, 1000), (5001, 600)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_loss_and_gradient(n, c, dt):
    rng = np.random.default_rng(n * 13 + c)
    x = _logits(rng, n, c, dt)
    labels = rng.integers(0, c, n).astype(np.int32)
    if n > 4:
        labels[rng.random(n) < 0.1] = -1
    loss = torch.full((n,), 7.0, device="cuda")
    total = torch.full((2,), 7.0, device="cuda")
    grad = torch.full_like(x, 7.0)
    ws = _ws(n, c)
    for mean, gs in ((True, 1.0), (False, 0.25)):
        sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, grad, ws, mean=mean, grad_scale=gs)
        sg.sg_stream_check()
        _check(x, labels, loss, total, grad, mean, gs)
    first = (loss.clone(), total.clone(), grad.clone())
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, grad, ws, mean=False, grad_scale=0.25)
    sg.sg_stream_check()
    assert all(torch.equal(a, b) for a, b in zip(first, (loss, total, grad)))  # the same bits
    # loss alone, and in place
    only = torch.empty_like(loss)
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, only, None, None, ws, mean=False, grad_scale=0.25)
    inplace = x.clone()
    sg.sg_xent(inplace, torch.from_numpy(labels).cuda(), n, None, loss, total, inplace, ws, mean=False, grad_scale=0.25)
    sg.sg_stream_check()
    assert torch.equal(only, first[0]) and torch.equal(inplace, first[2])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", [(2000, 2500), (1100, 9001), (500, 20003), (470, 33000), (240, 60001), (300, 14000)])
def test_many_long_rows(n, c, dt):
    # more rows than the grid has clusters: rows follow one another in a cluster
    rng = np.random.default_rng(n + c)
    x = _logits(rng, n, c, dt)
    labels = rng.integers(0, c, n).astype(np.int32)
    labels[rng.random(n) < 0.15] = -1
    labels[-3:] = -1
    x[1, ::2] = float("-inf")
    x[2, :] = float("-inf")
    labels[1], labels[2] = 1, -1
    loss, total = torch.full((n,), 7.0, device="cuda"), torch.full((2,), 7.0, device="cuda")
    grad = torch.full_like(x, 7.0)
    ws = _ws(n, c)
    for m in (n, n - 101):
        d_n = None if m == n else torch.tensor([m], dtype=torch.int32, device="cuda")
        sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, d_n, loss, total, grad, ws)
        sg.sg_stream_check()
        _check(x, labels, loss, total, grad, True, 1.0, m)
    inplace = x.clone()
    sg.sg_xent(inplace, torch.from_numpy(labels).cuda(), n, None, loss, total, inplace, ws)
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, grad, ws)
    sg.sg_stream_check()
    assert torch.equal(inplace, grad)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("c,pad,shift", [(100, 4, 0), (100, 1, 1), (129, 0, 3), (1030, 5, 2), (9000, 3, 1),
                                         (20001, 0, 5), (64, 64, 8)])
def test_strides_and_alignment(dt, c, pad, shift):
    rng = np.random.default_rng(c + pad)
    n = 6

    def strided(p, s, fill):
        buf = torch.full((n * (c + p) + s + 8,), fill, dtype=DT[dt], device="cuda")
        return buf[s: s + n * (c + p)].view(n, c + p)[:, :c], buf
    x, xbuf = strided(pad, shift, float("nan"))  # what lies between the rows must not be used
    x.copy_(_logits(rng, n, c, dt))
    labels = rng.integers(0, c, n).astype(np.int32)
    for p, s in ((pad, shift), (pad + 1, 0), (0, 8)):
        grad, gbuf = strided(p, s, 7.0)
        loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
        sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, grad, _ws(n, c))
        sg.sg_stream_check()
        _check(x, labels, loss, total, grad, True, 1.0)
        kept = gbuf.clone()
        kept[s: s + n * (c + p)].view(n, c + p)[:, :c] = 7.0
        assert bool((kept == 7.0).all())
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, x, _ws(n, c))  # in place, strided
    sg.sg_stream_check()
    between = xbuf.clone()
    between[shift: shift + n * (c + pad)].view(n, c + pad)[:, :c] = float("nan")
    assert torch.equal(x, grad) and bool(torch.isnan(between).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("c", [40, 5000, 40000])
def test_masked_classes_and_empty_rows(dt, c):
    rng = np.random.default_rng(c)
    n = 8
    x = _logits(rng, n, c, dt)
    labels = rng.integers(0, c, n).astype(np.int32)
    ninf = float("-inf")
    x[0, ::2] = ninf
    x[0, int(labels[0])] = 1.0
    x[1, int(labels[1])] = ninf            # the label itself is masked
    x[2, :] = ninf                          # nothing is left
    x[3, :] = ninf
    x[3, int(labels[3])] = -3.0             # the label alone is left
    x[4, :] = torch.finfo(x.dtype).min      # the type's lowest value everywhere: uniform
    x[5, :] = torch.finfo(x.dtype).min
    x[5, c // 2] = 50.0
    x[6, :] = 80.0
    labels[7] = -1
    loss, total, grad = torch.empty(n, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, grad, _ws(n, c))
    sg.sg_stream_check()
    keep = [0, 1, 2, 3, 4, 6, 7] if labels[5] != c // 2 else list(range(n))
    lo, lerr, _, valid, gr, err = _reference(x.double().cpu().numpy(), labels, True, 1.0)
    got, g = loss.double().cpu().numpy(), grad.double().cpu().numpy()
    for r in keep:
        if np.isinf(lo[r]):
            assert np.isposinf(got[r])
        else:
            assert abs(got[r] - lo[r]) <= lerr[r]
        assert np.all(within(g[r], gr[r], err[r], dt == "bf16"))
    assert got[5] > 1e38 or labels[5] == c // 2
    assert float(total[1]) == valid and np.isposinf(float(total[0]))
    assert not bool(torch.isnan(grad).any())
    assert bool((grad[2] == 0).all()) and bool((grad[7] == 0).all()) and got[7] == 0.0


@pytest.mark.parametrize("c", [40, 5000, 40000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_inf_stay_in_their_row(c, bad):
    rng = np.random.default_rng(c)
    n = 5
    x = _logits(rng, n, c, "f32")
    labels = rng.integers(0, c, n).astype(np.int32)
    labels[4] = -1
    x[1, c // 3] = bad
    x[3, :] = float("-inf")
    x[3, 0] = float("nan")
    x[4, 1] = bad                           # an ignored row: not looked at
    loss, total, grad = torch.empty(n, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, grad, _ws(n, c))
    sg.sg_stream_check()
    assert bool(torch.isnan(loss[1])) and bool(torch.isnan(loss[3])) and bool(torch.isnan(total[0]))
    assert bool(torch.isfinite(loss[[0, 2, 4]]).all()) and bool(torch.isfinite(grad[[0, 2, 4]]).all())
    assert bool((grad[4] == 0).all())


@pytest.mark.parametrize("n", [0, 1, 100, 6000])
@pytest.mark.parametrize("c", [20, 3000])
def test_device_count(n, c):
    rng = np.random.default_rng(n + c)
    n_cap = 6000 if c == 20 else 150
    n = min(n, n_cap)
    x = _logits(rng, n_cap, c, "f32")
    x[n:] = float("nan")
    labels = rng.integers(-1, c, n_cap).astype(np.int32)
    loss = torch.full((n_cap,), 7.0, device="cuda")
    total, grad = torch.empty(2, device="cuda"), torch.full_like(x, 7.0)
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n_cap, torch.tensor([n], dtype=torch.int32, device="cuda"), loss,
               total, grad, _ws(n_cap, c))
    sg.sg_stream_check()
    if n:
        _check(x, labels, loss, total, grad, True, 1.0, n)
    else:
        assert total.tolist() == [0.0, 0.0]
    assert bool((loss[n:] == 7.0).all()) and bool((grad[n:] == 7.0).all())


def test_no_rows_and_no_labels():
    c = 50
    total = torch.full((2,), 7.0, device="cuda")
    x = torch.zeros((0, c), device="cuda")
    sg.sg_xent(x, torch.zeros(0, dtype=torch.int32, device="cuda"), 0, None, torch.zeros(0, device="cuda"), total, x,
               _ws(1, c))
    sg.sg_stream_check()
    assert total.tolist() == [0.0, 0.0]
    x = torch.randn((4, c), device="cuda")
    grad, loss = torch.full_like(x, 7.0), torch.full((4,), 7.0, device="cuda")
    sg.sg_xent(x, torch.full((4,), -1, dtype=torch.int32, device="cuda"), 4, None, loss, total, grad, _ws(4, c))
    sg.sg_stream_check()
    assert total.tolist() == [0.0, 0.0] and not bool(grad.any()) and not bool(loss.any())


@pytest.mark.parametrize("c", [30, 9000])
def test_bad_label_is_reported_and_ignored(c):
    x = torch.randn((3, c), device="cuda")
    grad, loss, total = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(2, device="cuda")
    sg.sg_xent(x, torch.tensor([1, c, -2], dtype=torch.int32, device="cuda"), 3, None, loss, total, grad, _ws(3, c))
    with pytest.raises(sg.SgError) as e:
        sg.sg_stream_check()
    assert e.value.status == sg.SG_ERR_INVALID_INDEX
    assert float(total[1]) == 3.0 and not bool(grad[1:].any()) and loss[1:].tolist() == [0.0, 0.0]


@pytest.mark.parametrize("n,c", [(12, 60), (3, 7000)])
def test_gradient_against_differences(n, c):
    # central differences of the mean loss along random directions: with step
    # h = 2^-6 the truncation is h^2 / 6 times a third derivative (below 8 for
    # |direction| <= 2), the losses' rounding 2^-20 / h
    rng = np.random.default_rng(c)
    x = _logits(rng, n, c, "f32")
    labels = torch.from_numpy(rng.integers(0, c, n).astype(np.int32)).cuda()
    loss, total, grad = torch.empty(n, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
    sg.sg_xent(x, labels, n, None, loss, total, grad, _ws(n, c))
    h = 2.0 ** -6
    for k in range(4):
        d = torch.from_numpy(rng.uniform(-2, 2, (n, c)).astype(np.float32)).cuda()
        f = []
        for s in (h, -h):
            sg.sg_xent(x + s * d, labels, n, None, loss, total, None, _ws(n, c))
            f.append(float(loss.double().sum()) / n)
        want = (f[0] - f[1]) / (2 * h)
        got = float((grad.double() * d.double()).sum())
        assert abs(got - want) <= h * h / 6 * 8 + 2.0 ** -20 / h


def test_other_stream_and_graph_replay():
    rng = np.random.default_rng(1)
    n, c = 200, 300
    s = torch.cuda.Stream()
    x = _logits(rng, n, c, "f32")
    labels = torch.zeros(n, dtype=torch.int32, device="cuda")
    loss, total, grad = torch.empty(n, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
    ws = _ws(n, c)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        sg.sg_xent(x, labels, n, None, loss, total, grad, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        sg.sg_xent(x, labels, n, None, loss, total, grad, ws)
    for _ in range(2):
        h = rng.integers(-1, c, n).astype(np.int32)
        labels.copy_(torch.from_numpy(h))
        x.copy_(_logits(rng, n, c, "f32"))
        graph.replay()
        torch.cuda.synchronize()
        _check(x, h, loss, total, grad, True, 1.0)
    sg.sg_stream_check()
