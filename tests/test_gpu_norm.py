"""Layer norm and its gradient (sg_layernorm_fwd, sg_layernorm_bwd) against
torch in 64 bits.

Tolerances (u = 2^-24): a row's sums are taken 16 values at a time in a thread and
then by halves (10 levels at most): off by 26 u of the sum of absolute values.  So
the mean is off by 28 u mean|x|, the variance by 32 u of itself and the mean's error
squared, 1 / deviation by 18 u, and y by |w| (r 28 u mean|x| + 24 u |h|) + 2 u (|y| + |b|).
Backward (mean and rstd are inputs): h is off by 2 u |h|, u = g w by u, the means of u
and u h by 32 u of the means of |u| and |u h|, and dx by
r (4 |u| + 34 mean|u| + 38 |h| mean|u h|) u.  A column's sum over the rows is taken over
a thread's rows, then the groups', then the blocks': at most rows / 8 + 64 in a row, fewer
than n / 8 + 128, of values off by 4 u.  bf16 results have to be the rounding of a
value within that."""
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_xent_rows import _rounded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


class _Guarded:
    """A workspace of exactly the bytes asked for, with bytes behind it that
    have to stay as they are."""
    def __init__(self, n, d):
        need = sg.sg_layernorm_bwd_workspace(n, d)
        self.all = sg.aligned_workspace(need + (1 << 20))
        self.all.fill_(0xCD)
        self.ws, self.rest = self.all[:need], self.all[need:]

    def check(self):
        assert bool((self.rest == 0xCD).all())


def _ws(n, d):
    ws = sg.aligned_workspace(sg.sg_layernorm_bwd_workspace(n, d))
    ws.fill_(0xCD)
    return ws


def _within(got, want, tol):
    if got.dtype == torch.bfloat16:
        tol = tol + 1e-40
        ok = (_rounded(want - tol) <= got.double()) & (got.double() <= _rounded(want + tol))
    else:
        ok = (got.double() - want).abs() <= tol + 1e-44
    assert bool(ok.all()), (int((~ok).sum()), (got.double() - want)[~ok][:3], tol.expand_as(want)[~ok][:3])


def _inputs(n, d, dt, dw, seed, level=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn((n, d), generator=g, device="cuda") * 2 + level * torch.randn((n, 1), generator=g, device="cuda")).to(DT[dt])
    gr = torch.randn((n, d), generator=g, device="cuda").to(DT[dt])
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(DT[dw])
    b = (0.2 * torch.randn(d, generator=g, device="cuda")).to(DT[dw])
    return x, gr, w, b


def _hold_fwd(x, w, b, y, mean, rstd, eps=EPS):
    x64 = x.double()
    mu = x64.mean(1, keepdim=True)
    var = (x64 - mu).square().mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    h = (x64 - mu) * r
    w64 = torch.ones_like(h[0]) if w is None else w.double()
    b64 = torch.zeros_like(h[0]) if b is None else b.double()
    mag = x64.abs().mean(1, keepdim=True)
    off = 28 * U * mag  # of the mean
    rel = 24 * U + 0.5 * (off * r) ** 2
    want = h * w64 + b64
    _within(y, want, w64.abs() * (r * off + rel * h.abs()) + 2 * U * (want.abs() + b64.abs()))
    if mean is not None:
        assert bool(((mean.double() - mu[:, 0]).abs() <= off[:, 0] + 1e-44).all())
        assert bool(((rstd.double() - r[:, 0]).abs() <= (rel * r)[:, 0]).all())


def _hold_bwd(g, x, w, mean, rstd, dx, dw, db):
    n, d = x.shape
    g64, mu, r = g.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (x.double() - mu) * r
    u = g64 * (1 if w is None else w.double())
    want = r * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    tol = r * U * (4 * u.abs() + 34 * u.abs().mean(1, keepdim=True) + 38 * h.abs() * (u * h).abs().mean(1, keepdim=True))
    _within(dx, want, tol)
    if dw is not None:
        _within(dw, (g64 * h).sum(0), U * (n / 8 + 132) * (g64 * h).abs().sum(0))
    if db is not None:
        _within(db, g64.sum(0), U * (n / 8 + 128) * g64.abs().sum(0))


def _fwd(x, w, b, **kw):
    n = len(x)
    y, m, r = torch.full_like(x, 7.0), torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    sg.sg_layernorm_fwd(x, w, b, n, kw.pop("d_n", None), y, m, r, **kw)
    sg.sg_stream_check()
    return y, m, r


def _bwd(g, x, w, m, r, dtype_w=None, d_n=None):
    n, d = x.shape
    dx = torch.full_like(x, 7.0)
    dt = w.dtype if w is not None else dtype_w or torch.float32
    dw, db = torch.full((d,), 7.0, device="cuda", dtype=dt), torch.full((d,), 7.0, device="cuda", dtype=dt)
    guarded = _Guarded(n, d)
    sg.sg_layernorm_bwd(g, x, w, m, r, n, d_n, dx, dw, db, guarded.ws)
    sg.sg_stream_check()
    guarded.check()
    return dx, dw, db


# every form: groups of 4 to 32 lanes, blocks of 64 to 1024 threads; units of 16 down to 2 bytes
DIMS = [1, 2, 3, 4, 8, 12, 16, 20, 31, 32, 33, 48, 64, 65, 96, 100, 127, 128, 130, 200, 250, 256, 257, 300, 500, 511, 512, 514, 602,
        1000, 1001, 1024, 1026, 1028, 1500, 2047, 2048, 2050, 2500, 4095, 4096, 4098, 5000, 8190, 8192, 8193, 10000, 16383, 16384]


@pytest.mark.parametrize("dt,dw", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("d", DIMS)
def test_forward_and_gradient(d, dt, dw):
    for n in (1, 2, 37, 300 if d > 2000 else 3001):
        x, g, w, b = _inputs(n, d, dt, dw, n + d)
        y, m, r = _fwd(x, w, b)
        _hold_fwd(x, w, b, y, m, r)
        got = _bwd(g, x, w, m, r)
        _hold_bwd(g, x, w, m, r, *got)
    again = _fwd(x, w, b) + _bwd(g, x, w, m, r)
    assert all(torch.equal(a, c) for a, c in zip((y, m, r) + got, again))  # the same bits
    # in place
    z = x.clone()
    sg.sg_layernorm_fwd(z, w, b, n, None, z)
    assert torch.equal(z, y)
    for over in (0, 1):
        gg, xx = g.clone(), x.clone()
        dx = (gg, xx)[over]
        sg.sg_layernorm_bwd(gg, xx, w, m, r, n, None, dx, None, None, _ws(n, d))
        assert torch.equal(dx, got[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(200001, 64), (60001, 128), (30011, 1001), (9000, 4096), (3000, 8192), (2000, 16384), (100000, 7)])
def test_many_rows(n, d, dt):
    x, g, w, b = _inputs(n, d, dt, "f32", d)
    y, m, r = _fwd(x, w, b)
    _hold_fwd(x, w, b, y, m, r)
    _hold_bwd(g, x, w, m, r, *_bwd(g, x, w, m, r))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1200, 1300, 9700, 9800])
@pytest.mark.parametrize("d", [257, 300, 400, 513, 700, 1000])
def test_rows_enough_for_all_warps_or_not(n, d, dt):
    x, g, w, b = _inputs(n, d, dt, "f32", n + d)
    y, m, r = _fwd(x, w, b)
    _hold_fwd(x, w, b, y, m, r)
    _hold_bwd(g, x, w, m, r, *_bwd(g, x, w, m, r))


def test_two_streams_at_once():
    cases = [_inputs(5000, 1001, "bf16", "f32", 1), _inputs(3000, 4096, "f32", "bf16", 2), _inputs(900, 64, "f32", "f32", 3)]
    want, outs = [], []
    for x, g, w, b in cases:
        y, m, r = _fwd(x, w, b)
        want.append((y, m, r) + _bwd(g, x, w, m, r))
        outs.append([torch.empty_like(t) for t in want[-1]])
    ws = [_ws(*c[0].shape) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for (x, g, w, b), o, s, m in zip(cases, outs, streams, ws):
            with torch.cuda.stream(s):
                sg.sg_layernorm_fwd(x, w, b, len(x), None, *o[:3])
                sg.sg_layernorm_bwd(g, x, w, o[1], o[2], len(x), None, *o[3:], m)
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [5, 64, 100, 700, 4096])
def test_without_parameters_and_parts(d, dt):
    x, g, w, b = _inputs(50, d, dt, "f32", d)
    y, m, r = _fwd(x, None, None)
    _hold_fwd(x, None, None, y, m, r)
    _hold_fwd(x, w, None, *_fwd(x, w, None))
    _hold_fwd(x, None, b, *_fwd(x, None, b))
    got = _bwd(g, x, None, m, r)
    _hold_bwd(g, x, None, m, r, *got)
    for one in (0, 1):
        dx, part = torch.empty_like(x), torch.empty(d, device="cuda")
        sg.sg_layernorm_bwd(g, x, None, m, r, 50, None, dx, (part, None)[one], (None, part)[one], _ws(50, d))
        assert torch.equal(dx, got[0]) and torch.equal(part, got[1 + one])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1, 7, 64, 100, 300, 1001, 5000])
def test_far_levels_and_equal_values(d, dt):
    # rows far from zero, of equal values, of one value that stands out, of tiny values
    x, g, w, b = _inputs(12, d, dt, "f32", d, level=300.0)
    x[1], x[2], x[3, :] = 5.0, 0.0, x[3] * 1e-6
    x[4, d // 2] = 1000.0
    y, m, r = _fwd(x, w, b)
    _hold_fwd(x, w, b, y, m, r)
    _hold_bwd(g, x, w, m, r, *_bwd(g, x, w, m, r))
    y, m, r = _fwd(x, w, b, eps=1e-2)
    _hold_fwd(x, w, b, y, m, r, eps=1e-2)


@pytest.mark.parametrize("d", [20, 300, 3000])
def test_nan_stays_in_its_row(d):
    x, g, w, b = _inputs(20, d, "f32", "f32", d)
    y, m, r = _fwd(x, w, b)
    dx, _, _ = _bwd(g, x, w, m, r)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[7, d // 2] = bad
        y2, m2, r2 = _fwd(z, w, b)
        keep = torch.arange(20, device="cuda") != 7
        assert bool(torch.isnan(y2[7]).all()) and torch.equal(y2[keep], y[keep])
        dx2, dw2, _ = _bwd(g, z, w, m2, r2)
        assert torch.equal(dx2[keep], dx[keep]) and bool(torch.isnan(dw2).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [4, 64, 100, 128, 1001, 4096])
@pytest.mark.parametrize("start,gap", [(0, 8), (1, 0), (2, 2), (4, 12)])
def test_strides_and_rows_behind_the_count(d, start, gap, dt):
    n = 45
    x, g, w, b = _inputs(n, d, dt, "f32", d)

    def place(t):
        wide = torch.full((n, start + d + gap), 7.0, dtype=t.dtype, device="cuda")
        wide[:, start:start + d] = t
        return wide, wide[:, start:start + d]
    wide_w = torch.full((d + 3,), 7.0, device="cuda")
    wide_w[1:1 + d] = w
    for count in (17, 0, n + 1):
        d_n = torch.tensor([count], dtype=torch.int32, device="cuda")
        r_ = min(count, n)
        (_, xs), (_, gs), (yw, ys), (dw_, ds) = place(x), place(g), place(torch.full_like(x, 7.0)), place(torch.full_like(x, 7.0))
        m, r = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
        sg.sg_layernorm_fwd(xs, wide_w[1:1 + d], b, n, d_n, ys, m, r)
        sg.sg_stream_check()
        _hold_fwd(x[:r_], w, b, ys[:r_], m[:r_], r[:r_])
        pw, pb = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
        sg.sg_layernorm_bwd(gs, xs, wide_w[1:1 + d], m, r, n, d_n, ds, pw, pb, _ws(n, d))
        sg.sg_stream_check()
        _hold_bwd(g[:r_], x[:r_], w, m[:r_], r[:r_], ds[:r_], pw, pb)
        for t in (yw, dw_):
            t = t.clone()
            t[:r_, start:start + d] = 7.0
            assert bool((t == 7).all())
        assert bool((m[r_:] == 7).all()) and bool((r[r_:] == 7).all())


def test_no_rows():
    d = 40
    x = torch.empty((0, d), device="cuda")
    dw, db = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    e = torch.empty(0, device="cuda")
    sg.sg_layernorm_fwd(x, None, None, 0, None, x, e, e)
    sg.sg_layernorm_bwd(x, x, None, e, e, 0, None, x, dw, db, _ws(0, d))
    sg.sg_stream_check()
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_gradient_is_the_slope():
    # central differences in 64 bits: the third derivative of y in one x is below 100 r^3,
    # so a step of 1e-4 leaves below 1e-6 of the sums here
    n, d, h = 3, 11, 1e-4
    x, g, w, b = _inputs(n, d, "f32", "f32", 4)
    y, m, r = _fwd(x, w, b)
    dx, dw, db = _bwd(g, x, w, m, r)

    def f(x_, w_, b_):
        return (torch.nn.functional.layer_norm(x_, (d,), w_, b_, EPS) * g.double()).sum(1)
    x64, w64, b64 = x.double(), w.double(), b.double()
    for c in range(d):
        e = torch.zeros(d, dtype=torch.float64, device="cuda")
        e[c] = h
        assert float(((f(x64 + e, w64, b64) - f(x64 - e, w64, b64)) / (2 * h) - dx[:, c]).abs().max()) <= 1e-4
        assert abs(float((f(x64, w64 + e, b64) - f(x64, w64 - e, b64)).sum() / (2 * h) - dw[c])) <= 1e-4
        assert abs(float((f(x64, w64, b64 + e) - f(x64, w64, b64 - e)).sum() / (2 * h) - db[c])) <= 1e-4


def test_offsets_past_32_bits():
    n, d = 550000, 4096
    x = torch.empty((n, d), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    y, m, r = _fwd(x, None, None)
    at = torch.tensor([0, 1, 300000, 524287, 524288, n - 1], device="cuda")
    _hold_fwd(x[at], None, None, y[at], m[at], r[at])
    sg.sg_layernorm_bwd(y, x, None, m, r, n, None, y, None, None, _ws(n, d))  # g = y, replaced
    sg.sg_stream_check()
    g = _fwd(x[at].contiguous(), None, None)[0]
    _hold_bwd(g, x[at], None, m[at], r[at], y[at], None, None)


def test_two_graphs_share_a_workspace():
    cases = [_inputs(500, 64, "f32", "f32", 1), _inputs(300, 1001, "bf16", "f32", 2), _inputs(200, 4096, "bf16", "bf16", 3)]
    ws = sg.aligned_workspace(max(sg.sg_layernorm_bwd_workspace(len(c[0]), c[0].shape[1]) for c in cases))
    want, outs, graphs = [], [], []
    for x, g, w, b in cases:
        y, m, r = _fwd(x, w, b)
        want.append((y, m, r) + _bwd(g, x, w, m, r))
        outs.append([torch.empty_like(t) for t in want[-1]])
    torch.cuda.synchronize()
    for (x, g, w, b), o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sg.sg_layernorm_fwd(x, w, b, len(x), None, *o[:3])
            sg.sg_layernorm_bwd(g, x, w, o[1], o[2], len(x), None, *o[3:], ws)
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs + graphs[::-1]:
            graph.replay()
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))
