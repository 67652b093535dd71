"""Learned embeddings (sg_embed_fwd, sg_embed_bwd) against plain numpy in 64
bits.

Tolerances follow the arithmetic (u = 2^-24): the lookup is one fp32 product
(u); a sum of k rows is off by at most k u times the sum of |terms|, its
scaling by u, the addition into given rows by u of both parts.  A bf16 output
has to be the rounding of a value within that tolerance."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from rounding import within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
MODES = {"rows": sg.SG_GRAD_ROWS, "dense": sg.SG_GRAD_DENSE, "add": sg.SG_GRAD_ADD}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _f64(t):
    return t.double().cpu().numpy()


def _strided(rows, cols, dtype, pad, shift, fill=7.0):
    """A rows x cols device matrix whose rows are cols + pad elements apart
    and whose first element is `shift` elements past an aligned address;
    returns (view, the whole buffer)."""
    buf = torch.full((rows * (cols + pad) + shift + 8,), fill, dtype=dtype, device="cuda")
    view = buf[shift: shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return view, buf


def _ids(rng, n, n_rows, kind):
    if kind == "same":
        return np.full(n, n_rows - 1, np.int32)
    if kind == "none":
        return np.full(n, -1, np.int32)
    if kind == "sorted":
        return np.sort(rng.integers(0, n_rows, n)).astype(np.int32)
    if kind == "distinct":
        return rng.permutation(n_rows)[:n].astype(np.int32)
    v = np.minimum(n_rows - 1, np.floor((n_rows + 1) ** rng.random(n)) - 1).astype(np.int32)  # a power law
    v[rng.random(n) < 0.05] = -1
    return v


# ---------------------------------------------------------------- forward
@pytest.mark.parametrize("n,dim,n_rows,ti,to,pad,shift", [
    (1, 1, 1, "f32", "f32", 0, 0), (300, 64, 1000, "f32", "f32", 0, 0), (257, 100, 90, "f32", "bf16", 0, 0),
    (1000, 128, 5000, "bf16", "bf16", 0, 0), (333, 100, 777, "bf16", "f32", 0, 0), (65, 33, 100, "bf16", "bf16", 0, 0),
    (65, 33, 100, "f32", "f32", 1, 1), (70, 64, 100, "bf16", "f32", 3, 1), (70, 64, 100, "f32", "f32", 4, 4),
    (4097, 1030, 50, "f32", "bf16", 0, 0), (50001, 8, 3, "bf16", "f32", 0, 0)])
def test_lookup(n, dim, n_rows, ti, to, pad, shift):
    rng = np.random.default_rng(n + dim)
    table, _ = _strided(n_rows, dim, DT[ti], pad, shift)
    table.copy_(torch.from_numpy(rng.standard_normal((n_rows, dim)).astype(np.float32)))
    ids = _ids(rng, n, n_rows, "power")
    out, buf = _strided(n + 2, dim, DT[to], pad, shift)
    scale = 1.7
    sg.sg_embed_fwd(table, torch.from_numpy(ids).cuda(), n, None, scale, out)
    sg.sg_stream_check()
    want = _f64(table)[np.maximum(ids, 0)] * np.float64(np.float32(scale)) * (ids >= 0)[:, None]
    assert np.all(within(_f64(out[:n]), want, U * np.abs(want), to == "bf16"))
    # nothing outside the rows was written
    kept = buf.clone()
    kept[shift: shift + (n + 2) * (dim + pad)].view(n + 2, dim + pad)[:n, :dim] = 7.0
    assert bool((kept == 7.0).all())


def test_lookup_device_count_and_bad_id():
    table = torch.arange(40.0, device="cuda").view(10, 4)
    ids = torch.tensor([3, 9, -1, 10, -5, 2], dtype=torch.int32, device="cuda")
    for n in (0, 2, 6, 9):  # 9: above the capacity, clamped
        out = torch.full((6, 4), 7.0, device="cuda")
        sg.sg_embed_fwd(table, ids, 6, torch.tensor([n], dtype=torch.int32, device="cuda"), 2.0, out)
        m = min(n, 6)
        if m == 6:
            with pytest.raises(sg.SgError) as e:
                sg.sg_stream_check()
            assert e.value.status == sg.SG_ERR_INVALID_INDEX
        else:
            sg.sg_stream_check()
        want = torch.full((6, 4), 7.0)
        for i, v in enumerate([3, 9, -1, 10, -5, 2][:m]):
            want[i] = 2 * torch.arange(4.0) + 8 * v if 0 <= v < 10 else 0.0
        assert torch.equal(out.cpu(), want)
    sg.sg_embed_fwd(table, ids, 0, None, 1.0, torch.empty((0, 4), device="cuda"))
    sg.sg_stream_check()


def test_lookup_past_31_bit_offsets():
    n_rows, dim = 17_000_003, 128  # 2.18e9 elements
    table = torch.empty((n_rows, dim), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([n_rows - 1, 0, 16_777_217, 9], dtype=torch.int32, device="cuda")
    rows = torch.randn((4, dim), device="cuda").bfloat16()
    table[ids.long()] = rows
    out = torch.empty((4, dim), dtype=torch.bfloat16, device="cuda")
    sg.sg_embed_fwd(table, ids, 4, None, 1.0, out)
    sg.sg_stream_check()
    assert torch.equal(out, rows)
    # and the gradient added at such offsets
    ws = sg.aligned_workspace(sg.sg_embed_bwd_workspace(4, n_rows, dim, sg.SG_GRAD_ADD))
    g = torch.ones((4, dim), device="cuda")
    sg.sg_embed_bwd(ids, 4, None, n_rows, g, -1.0, table, sg.SG_GRAD_ADD, ws)
    sg.sg_stream_check()
    assert torch.equal(table[ids.long()], (rows.float() - 1.0).bfloat16())


# --------------------------------------------------------------- backward
def _bwd(ids, n_rows, g, scale, mode, to, base=None, n=None, out_view=None):
    """Runs sg_embed_bwd; returns (rows or None, gradient rows as float64)."""
    n_cap, dim = len(ids), g.shape[1]
    m = MODES[mode]
    ws = sg.aligned_workspace(sg.sg_embed_bwd_workspace(n_cap, n_rows, dim, m))
    ws.fill_(0xAB)
    d_n = None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")
    dev = torch.from_numpy(ids).cuda()
    if mode == "rows":
        grad = torch.full((n_cap, dim), 7.0, dtype=DT[to], device="cuda") if out_view is None else out_view
        rows = torch.full((n_cap,), -9, dtype=torch.int32, device="cuda")
        cnt = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        sg.sg_embed_bwd(dev, n_cap, d_n, n_rows, g, scale, grad, m, ws, rows=rows, n_out=cnt)
        sg.sg_stream_check()
        k = int(cnt.item())
        assert bool((rows[k:] == -9).all()) and bool((grad[k:] == 7.0).all())
        return rows[:k].cpu().numpy(), _f64(grad[:k])
    grad = torch.full((n_rows, dim), 7.0, dtype=DT[to], device="cuda") if out_view is None else out_view
    if mode == "add":
        grad.copy_(base)
    sg.sg_embed_bwd(dev, n_cap, d_n, n_rows, g, scale, grad, m, ws)
    sg.sg_stream_check()
    return None, _f64(grad)


def _reference(ids, n_rows, g, scale):
    """(sums, sums of |terms|, counts) per table row, in 64 bits."""
    g = _f64(g) * np.float64(np.float32(scale))
    at = np.nonzero(ids >= 0)[0]
    s, a = np.zeros((n_rows, g.shape[1])), np.zeros((n_rows, g.shape[1]))
    np.add.at(s, ids[at], g[at])
    np.add.at(a, ids[at], np.abs(g[at]))
    return s, a, np.bincount(ids[at], minlength=n_rows)


def _check_bwd(got, ids, n_rows, g, scale, mode, to, base=None):
    rows, grad = got
    s, a, k = _reference(ids, n_rows, g, scale)
    tol = (k[:, None] + 2) * U * a
    want = s
    if mode == "rows":
        ids_want = np.nonzero(k)[0]
        assert np.array_equal(rows, ids_want)
        want, tol = s[ids_want], tol[ids_want]
    if mode == "add":
        want = s + _f64(base)
        tol = tol + U * (np.abs(s) + np.abs(_f64(base))) * (k[:, None] > 0)
    assert grad.shape == want.shape
    assert np.all(within(grad, want, tol, to == "bf16"))


@pytest.mark.parametrize("mode", ["rows", "dense", "add"])
@pytest.mark.parametrize("n,dim,n_rows,kind,tg,to", [
    (1, 1, 1, "same", "f32", "f32"), (31, 4, 7, "power", "f32", "f32"), (33, 3, 5, "power", "bf16", "f32"),
    (300, 64, 1000, "power", "f32", "f32"), (4096, 100, 255, "power", "f32", "bf16"),
    (4097, 100, 256, "sorted", "bf16", "bf16"), (8193, 8, 257, "power", "bf16", "f32"),
    (1000, 33, 3000, "distinct", "f32", "f32"), (777, 130, 65535, "power", "f32", "f32"),
    (20000, 256, 65536, "power", "f32", "f32"), (3000, 1024, 40, "power", "bf16", "bf16"),
    (70001, 8, 9, "same", "f32", "f32"), (70001, 12, 2, "sorted", "bf16", "f32"), (500, 20, 300, "none", "f32", "f32"),
    (40000, 32, 1, "same", "f32", "f32"), (66000, 64, 500, "power", "f32", "f32"),
    (16384, 16, 70000, "power", "f32", "f32"), (16385, 20, 3000, "sorted", "f32", "f32"), (32768, 8, 1 << 20, "power", "bf16", "f32"), (30000, 12, 300, "same", "f32", "f32"),
    (65536, 8, 20000, "power", "f32", "bf16"), (131072, 4, 100000, "power", "f32", "f32"),
    (131073, 4, 256, "sorted", "bf16", "f32"), (140000, 20, 5000, "none", "f32", "f32"),
    (700001, 4, 3000, "power", "f32", "f32"), (650000, 40, 2, "same", "bf16", "f32")])
def test_gradient(n, dim, n_rows, kind, tg, to, mode):
    rng = np.random.default_rng(n * 7 + dim)
    ids = _ids(rng, n, n_rows, kind)
    g = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).cuda().to(DT[tg])
    base = torch.from_numpy(rng.standard_normal((n_rows, dim)).astype(np.float32)).cuda().to(DT[to])
    got = _bwd(ids, n_rows, g, -0.3, mode, to, base)
    _check_bwd(got, ids, n_rows, g, -0.3, mode, to, base)
    again = _bwd(ids, n_rows, g, -0.3, mode, to, base)  # one order of summation: the same bits
    assert np.array_equal(got[1], again[1])


@pytest.mark.parametrize("mode", ["rows", "dense"])
@pytest.mark.parametrize("kind", ["power", "same", "distinct"])
@pytest.mark.parametrize("n", [1023, 1024, 1025, 2048, 3071, 3073, 4095, 8191, 8192])
def test_gradient_where_the_sort_changes(n, kind, mode):
    # the largest lists of one form of the sort and the shortest of the next
    rng = np.random.default_rng(n)
    dim, n_rows = 8, 9000
    ids = _ids(rng, n, n_rows, kind)
    g = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).cuda()
    base = torch.zeros((n_rows, dim), device="cuda")
    _check_bwd(_bwd(ids, n_rows, g, 1.5, mode, "f32", base), ids, n_rows, g, 1.5, mode, "f32", base)
    part = n * 2 // 3  # fewer, counted on the device
    g[part:] = float("nan")
    _check_bwd(_bwd(ids, n_rows, g, 1.5, mode, "f32", base, n=part), ids[:part], n_rows, g[:part], 1.5, mode, "f32", base)


@pytest.mark.parametrize("mode", ["rows", "dense", "add"])
def test_gradient_wide_ids_and_sort_passes(mode):
    # IDs across all four digits of the sort where the table can be that long
    rng = np.random.default_rng(5)
    n, dim, n_rows = 5000, 4, 20_000_000 if mode == "rows" else 300_000
    ids = rng.integers(0, n_rows, n).astype(np.int32)
    ids[:100] = n_rows - 1 - np.arange(100) // 2
    g = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).cuda()
    if mode != "rows":
        base = torch.zeros((n_rows, dim), device="cuda")
        _check_bwd(_bwd(ids, n_rows, g, 1.0, mode, "f32", base), ids, n_rows, g, 1.0, mode, "f32", base)
        return
    rows, grad = _bwd(ids, n_rows, g, 1.0, mode, "f32")
    uniq, inv = np.unique(ids, return_inverse=True)
    s, a = np.zeros((len(uniq), dim)), np.zeros((len(uniq), dim))
    np.add.at(s, inv, _f64(g))
    np.add.at(a, inv, np.abs(_f64(g)))
    assert np.array_equal(rows, uniq)
    assert np.all(np.abs(grad - s) <= (np.bincount(inv)[:, None] + 2) * U * a)


@pytest.mark.parametrize("mode", ["rows", "dense", "add"])
@pytest.mark.parametrize("n", [0, 1, 64, 4096, 5000, 9000])
def test_gradient_device_count(mode, n):
    rng = np.random.default_rng(n)
    n_cap, dim, n_rows = 9000, 24, 400
    ids = _ids(rng, n_cap, n_rows, "power")
    g = torch.from_numpy(rng.standard_normal((n_cap, dim)).astype(np.float32)).cuda()
    g[n:] = float("nan")  # rows past the count take no part
    base = torch.ones((n_rows, dim), device="cuda")
    _check_bwd(_bwd(ids, n_rows, g, 0.5, mode, "f32", base, n=n), ids[:n], n_rows, g[:n], 0.5, mode, "f32", base)


@pytest.mark.parametrize("mode", ["rows", "dense", "add"])
@pytest.mark.parametrize("dim,pad,shift,tg,to", [(64, 4, 4, "f32", "f32"), (64, 1, 0, "f32", "f32"),
                                                 (40, 3, 1, "bf16", "bf16"), (64, 8, 8, "bf16", "f32"),
                                                 (64, 4, 4, "bf16", "bf16")])
def test_gradient_strides_and_alignment(mode, dim, pad, shift, tg, to):
    rng = np.random.default_rng(dim + pad)
    n, n_rows = 700, 90
    ids = _ids(rng, n, n_rows, "power")
    g, _ = _strided(n, dim, DT[tg], pad, shift)
    g.copy_(torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)))
    rows_out = n if mode == "rows" else n_rows
    view, buf = _strided(rows_out, dim, DT[to], pad, shift)
    base = torch.ones((n_rows, dim), dtype=DT[to], device="cuda")
    _check_bwd(_bwd(ids, n_rows, g, 1.0, mode, to, base, out_view=view), ids, n_rows, g, 1.0, mode, to, base)
    kept = buf.clone()
    kept[shift: shift + rows_out * (dim + pad)].view(rows_out, dim + pad)[:, :dim] = 7.0
    assert bool((kept == 7.0).all())  # the gaps between rows were not written


def test_gradient_is_the_adjoint_of_the_lookup():
    # the lookup is linear in the table, so its difference along any direction
    # D is exact: <g, lookup(D)> = <gradient, D>
    rng = np.random.default_rng(2)
    n, dim, n_rows = 3000, 48, 200
    ids = _ids(rng, n, n_rows, "power")
    g = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).cuda()
    d = torch.from_numpy(rng.standard_normal((n_rows, dim)).astype(np.float32)).cuda()
    out = torch.empty((n, dim), device="cuda")
    sg.sg_embed_fwd(d, torch.from_numpy(ids).cuda(), n, None, 3.0, out)
    _, grad = _bwd(ids, n_rows, g, 3.0, "dense", "f32")
    left, right = float((_f64(g) * _f64(out)).sum()), float((grad * _f64(d)).sum())
    size = float((np.abs(_f64(g)) * np.abs(_f64(out))).sum())
    assert abs(left - right) <= (np.bincount(ids[ids >= 0]).max() + 4) * U * size


def test_gradient_bad_id_is_reported_and_skipped():
    ids = np.array([1, 5, 1, -7, 0], np.int32)
    g = torch.ones((5, 4), device="cuda")
    for mode in MODES:
        with pytest.raises(sg.SgError) as e:
            _bwd(ids, 5, g, 1.0, mode, "f32", torch.zeros((5, 4), device="cuda"))
        assert e.value.status == sg.SG_ERR_INVALID_INDEX
    sg.sg_stream_check()


def test_other_stream_and_graph_replay():
    rng = np.random.default_rng(9)
    n, dim, n_rows = 5000, 32, 500
    s = torch.cuda.Stream()
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    g = torch.empty((n, dim), device="cuda")
    grad = torch.empty((n_rows, dim), device="cuda")
    ws = sg.aligned_workspace(sg.sg_embed_bwd_workspace(n, n_rows, dim, sg.SG_GRAD_DENSE))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        sg.sg_embed_bwd(ids, n, None, n_rows, g, 1.0, grad, sg.SG_GRAD_DENSE, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        sg.sg_embed_bwd(ids, n, None, n_rows, g, 1.0, grad, sg.SG_GRAD_DENSE, ws)
    for _ in range(2):
        h = _ids(rng, n, n_rows, "power")
        ids.copy_(torch.from_numpy(h))
        g.copy_(torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        sg.sg_stream_check()
        _check_bwd((None, _f64(grad)), h, n_rows, g, 1.0, "dense", "f32")
