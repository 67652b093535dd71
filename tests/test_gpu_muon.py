"""Newton-Schulz orthogonalisation and the Muon step (sg_orthogonalise,
sg_muon_step) against plain numpy in 64 bits.

Tolerance.  The operands of the products carry 22 bits and the sums 24, so a
step's products bring in an error of at most g = 32 * 2^-22 of ||X||_F: the
polynomial's parts a X, b A X, c A A X weigh |a| + 3 |b| + 5 |c| < 32 for
singular values up to about 1.1.  A later step multiplies an error by at most
|f'(t)| <= 4 over the singular values t that occur with the default
coefficients.  So after s steps ||error||_F <= g sum_k 4^(s - k) ||X_k||_F
(X_k: the iterates, k = 0: the normalised input).  bf16 output adds at most
half the spacing of bf16 numbers at each entry."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from rounding import quantum

pytestmark = pytest.mark.gpu
G = 32 * 2.0 ** -22
COEF = (3.4445, -4.7750, 2.0315)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _reference(u, steps=5, eps=1e-7, coef=None):
    """(orthogonalised matrix, bound on the Frobenius norm of the error)."""
    x = u / (np.linalg.norm(u) + np.float64(np.float32(eps)))
    if u.shape[0] > u.shape[1]:
        x = x.T
    err = G * np.linalg.norm(x)
    for k in range(steps):
        a, b, c = [np.float64(np.float32(v)) for v in (COEF if coef is None else coef[k])]
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
        err = 4 * err + G * np.linalg.norm(x)
    return (x.T if u.shape[0] > u.shape[1] else x), err


def _close(got, want, err, bf16, scale=1.0):
    d = np.abs(got - want)
    if bf16:
        d = np.maximum(0.0, d - 0.5 * quantum(np.maximum(np.abs(got), np.abs(want))))
    assert np.linalg.norm(d) <= abs(scale) * err


def _ws(count, rows, cols):
    ws = sg.aligned_workspace(sg.sg_orthogonalise_workspace(count, rows, cols))
    ws.fill_(0xEE)
    return ws


SHAPES = [(1, 1, 1), (1, 1, 300), (1, 5, 3), (1, 128, 128), (1, 128, 200), (2, 128, 256), (1, 128, 512),
          (1, 128, 2048), (1, 128, 2049), (1, 127, 129), (1, 64, 1000), (1, 16, 4096), (3, 33, 65), (1, 200, 128),
          (2, 256, 128), (1, 129, 130), (1, 130, 513), (1, 256, 256), (2, 257, 300), (1, 603, 401), (1, 100, 5000),
          (5, 128, 128), (1, 1024, 1000)]


@pytest.mark.parametrize("count,rows,cols", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_orthogonalise(count, rows, cols, dt):
    rng = np.random.default_rng(rows * 7 + cols)
    g = torch.from_numpy(rng.standard_normal((count, rows, cols)).astype(np.float32) * 1e-3).cuda().to(DT[dt])
    out = torch.full_like(g, 7.0)
    ws = _ws(count, rows, cols)
    sg.sg_orthogonalise(g, out, ws, scale=0.5)
    sg.sg_stream_check()
    for q in range(count):
        want, err = _reference(g[q].double().cpu().numpy())
        _close(out[q].double().cpu().numpy(), 0.5 * want, err, dt == "bf16", 0.5)
    first = out.clone()
    sg.sg_orthogonalise(g, g, ws, scale=0.5)  # in place, and the same bits again
    sg.sg_stream_check()
    assert torch.equal(first, g)


def test_singular_values_follow_the_polynomial():
    rng = np.random.default_rng(3)
    u, _ = np.linalg.qr(rng.standard_normal((96, 96)))
    v, _ = np.linalg.qr(rng.standard_normal((160, 96)))
    t = np.exp(np.linspace(0, -4, 96))
    g = torch.from_numpy(((u * t) @ v.T).astype(np.float32)).cuda()
    out = torch.empty_like(g)
    sg.sg_orthogonalise(g, out, _ws(1, 96, 160))
    sg.sg_stream_check()
    f = t / np.linalg.norm(t)
    for _ in range(5):
        f = COEF[0] * f + COEF[1] * f ** 3 + COEF[2] * f ** 5
    _, err = _reference(g.double().cpu().numpy())
    assert np.linalg.norm((u * f) @ v.T - out.double().cpu().numpy()) <= err + 485 * 2.0 ** -23  # g itself is rounded


@pytest.mark.parametrize("rows,cols", [(128, 200), (100, 90), (256, 300)])
@pytest.mark.parametrize("steps", [0, 1, 2, 7])
def test_steps_and_schedules(rows, cols, steps):
    rng = np.random.default_rng(steps)
    g = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).cuda()
    coef = [(1.5 + 0.2 * k, -0.5 - 0.05 * k, 0.01 * k) for k in range(steps)]
    out = torch.empty_like(g)
    sg.sg_orthogonalise(g, out, _ws(1, rows, cols), steps=steps, coef=coef if steps else None, eps=0.5)
    sg.sg_stream_check()
    want, err = _reference(g.double().cpu().numpy(), steps, 0.5, coef)
    _close(out.double().cpu().numpy(), want, err, False)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(128, 200, 3, 1), (128, 256, 8, 0), (40, 33, 1, 2), (300, 260, 5, 3),
                                                 (200, 100, 4, 4)])
def test_strides_and_alignment(rows, cols, pad, shift, dt):
    rng = np.random.default_rng(pad)

    def strided(fill):
        buf = torch.full((2 * rows * (cols + pad) + shift + 8,), fill, dtype=DT[dt], device="cuda")
        return buf[shift: shift + 2 * rows * (cols + pad)].view(2, rows, cols + pad)[:, :, :cols], buf
    g, _ = strided(float("nan"))
    g.copy_(torch.from_numpy(rng.standard_normal((2, rows, cols)).astype(np.float32)))
    out, buf = strided(7.0)
    sg.sg_orthogonalise(g, out, _ws(2, rows, cols))
    sg.sg_stream_check()
    for q in range(2):
        want, err = _reference(g[q].double().cpu().numpy())
        _close(out[q].double().cpu().numpy(), want, err, dt == "bf16")
    kept = buf.clone()
    kept[shift: shift + 2 * rows * (cols + pad)].view(2, rows, cols + pad)[:, :, :cols] = 7.0
    assert bool((kept == 7.0).all())


@pytest.mark.parametrize("rows,cols", [(128, 128), (100, 64), (300, 280)])
def test_zero_matrix_and_wide_range(rows, cols):
    g = torch.zeros((3, rows, cols), device="cuda")
    g[1] = torch.randn((rows, cols), device="cuda") * 1e12
    g[2] = torch.randn((rows, cols), device="cuda") * 1e-12
    out = torch.full_like(g, 7.0)
    sg.sg_orthogonalise(g, out, _ws(3, rows, cols), eps=1e-20)
    sg.sg_stream_check()
    assert not bool(out[0].any())
    for q in (1, 2):
        want, err = _reference(g[q].double().cpu().numpy(), eps=1e-20)
        _close(out[q].double().cpu().numpy(), want, err, False)


@pytest.mark.parametrize("count,rows,cols,dt", [(1, 128, 200, "f32"), (1, 128, 2048, "bf16"), (3, 128, 256, "bf16"),
                                                (2, 256, 128, "f32"), (1, 260, 333, "f32"), (1, 333, 260, "bf16"),
                                                (1, 1, 1, "f32"), (1, 7, 130, "bf16")])
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step(count, rows, cols, dt, nesterov):
    rng = np.random.default_rng(rows + cols)
    shape = (count, rows, cols)
    w = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) / 16).cuda().to(DT[dt])
    g = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * 1e-3).cuda()
    m = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * 1e-3).cuda()
    w2, m2 = torch.full_like(w, 7.0), torch.full_like(m, 7.0)
    lr, mu, wd, scale = 0.05, 0.9, 0.1, 1.25
    ws = _ws(count, rows, cols)
    kw = dict(lr=lr, momentum=mu, nesterov=nesterov, weight_decay=wd, scale=scale)
    sg.sg_muon_step(w, g, m, w2, m2, ws, **kw)
    sg.sg_stream_check()
    gd, md, wv = (t.double().cpu().numpy() for t in (g, m, w))
    muf = np.float64(np.float32(mu))
    m_new = muf * md + gd
    assert np.all(np.abs(m2.double().cpu().numpy() - m_new) <= 2.0 ** -23 * (np.abs(muf * md) + np.abs(gd)))
    u = gd + muf * m_new if nesterov else m_new
    for q in range(count):
        o, err = _reference(u[q])
        # the momentum update is rounded to fp32 before it is orthogonalised:
        # 2^-22 of ||u||, within the bound's factor for k = 0
        want = (1 - lr * wd) * wv[q] - lr * scale * o
        got = w2[q].double().cpu().numpy()
        d = np.maximum(0.0, np.abs(got - want) - 4 * 2.0 ** -24 * (np.abs(wv[q]) + np.abs(want)))
        if dt == "bf16":
            d = np.maximum(0.0, d - 0.5 * quantum(np.maximum(np.abs(got), np.abs(want))))
        assert np.linalg.norm(d) <= lr * scale * err * 1.01
    # in place gives the same bits
    sg.sg_muon_step(w, g, m, w, m, ws, **kw)
    sg.sg_stream_check()
    assert torch.equal(w, w2) and torch.equal(m, m2)


def test_other_stream_and_graph_replay():
    rng = np.random.default_rng(4)
    s = torch.cuda.Stream()
    g = torch.empty((128, 256), device="cuda")
    out = torch.empty_like(g)
    big = torch.empty((300, 260), device="cuda")
    big_out = torch.empty_like(big)
    ws, ws2 = _ws(1, 128, 256), _ws(1, 300, 260)
    g.normal_()
    big.normal_()
    torch.cuda.synchronize()

    def both():
        sg.sg_orthogonalise(g, out, ws)
        sg.sg_orthogonalise(big, big_out, ws2)
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for _ in range(2):
        for x in (g, big):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        for x, o in ((g, out), (big, big_out)):
            want, err = _reference(x.double().cpu().numpy())
            _close(o.double().cpu().numpy(), want, err, False)
    sg.sg_stream_check()
