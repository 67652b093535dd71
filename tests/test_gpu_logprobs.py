"""Log probabilities, entropy and top classes (sg_logprobs) against torch in 64
bits.

Tolerances (u = 2^-24, d = m - x, m the row's maximum): an exponential is off by
(8 + 2 d) u relative, 8 u more each time a thread's, warp's or CTA's sum is
brought to a larger maximum (at most once a 4,096 classes of a thread's part and 4
times to join them), and the sum of C of them by C / 256 u: the sum z by
e = (2 E[d] + C / 128 + 128) u relative, E[] the mean under the softmax.  A log
probability -d - log z is off by e, 2 u of either part and 8 u of the logarithm.
The entropy log z + E[d] is off by e, by E[d] e, by E[d (8 + 4 d + C / 128 + 64)] u
of the products' sum, and 8 u of either part.  The classes have to be exact."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _run(x, labels, k, n=None, d_n=None):
    rows = x.shape[0] if n is None else n
    out = [torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")]
    out += [torch.full((rows, k), 77, dtype=torch.int32, device="cuda"), torch.full((rows, k), 7.0, device="cuda")] if k \
        else [None, None]
    sg.sg_logprobs(x, labels, rows, d_n, out[0] if labels is not None else None, *out[1:])
    sg.sg_stream_check()
    return out


def _hold(x, labels, got, k):
    """Every row of the four outputs (rows without NaN and +inf)."""
    n, c = x.shape
    x64 = x.double()
    m = x64.amax(1, keepdim=True)
    none = m[:, 0] == -INF
    m = torch.where(none[:, None], torch.zeros_like(m), m)
    d = m - x64
    e = torch.exp(-d)
    z = e.sum(1)
    p = e / z.clamp(min=1e-300)[:, None]
    dd = torch.where(p > 0, d, torch.zeros_like(d))
    mean, square = (p * dd).sum(1), (p * dd * dd).sum(1)
    log_z = torch.where(none, torch.zeros_like(z), torch.log(z))
    err = U * (2 * mean + c / 128 + 128)
    logp, entropy, ids, top = got

    def near(a, want, tol, lost):
        a = a.double()
        far = lost & torch.isinf(want) | (want < -3.4e38)
        assert bool((a[far] == -INF).all() or (a[far] < -3.3e38).all())
        assert bool(((a - want).abs()[~far] <= tol[~far]).all()), float(((a - want).abs() / tol)[~far].max())
    if labels is not None:
        at = labels.long().clamp(min=0)
        dy = d.gather(1, at[:, None])[:, 0]
        want = torch.where(labels < 0, torch.zeros_like(dy), torch.where(none, torch.full_like(dy, -INF), -dy - log_z))
        near(logp, want, err + U * (2 * dy.clamp(max=1e300) + 10 * log_z + 4), torch.ones_like(none))
    want = torch.where(none, torch.zeros_like(mean), log_z + mean)
    tol = err * (1 + mean) + U * (72 * mean + 4 * square + c / 128 * mean + 8 * (log_z + mean))
    assert bool(((entropy.double() - want).abs() <= tol).all()), float(((entropy.double() - want).abs() / tol).max())
    if k:
        v, order = torch.sort(x64 + 0.0, dim=1, descending=True, stable=True)
        v, order = v[:, :k], order[:, :k]
        if k > c:
            v = torch.nn.functional.pad(v, (0, k - c), value=-INF)
            order = torch.nn.functional.pad(order, (0, k - c))
        gone = v == -INF
        want = torch.where(gone, torch.full_like(order, -1), order)
        assert torch.equal(ids.long(), want), (ids.long() != want).nonzero()[:4]
        dv = m - v
        near(top, torch.where(gone, v, -dv - log_z[:, None]),
             (err + U * 10 * log_z)[:, None] + U * (2 * dv.clamp(max=1e300) + 4), gone)


def _logits(n, c, dt, seed, spread=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (spread * torch.randn((n, c), generator=g, device="cuda")).to(DT[dt])


def _labels(n, c, seed):
    y = np.random.default_rng(seed).integers(-1, c, n).astype(np.int32)
    return torch.from_numpy(y).cuda()


SIZES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (5, 31, 40), (9, 32, 32), (256, 128, 5), (300, 47, 3), (2000, 47, 3), (129, 127, 64),
         (40, 129, 128), (33, 500, 20), (17, 513, 1), (40, 1000, 8), (17, 1025, 128), (9, 4097, 20), (7, 8191, 64),
         (600, 8193, 20), (4, 16385, 5), (3, 50257, 20), (700, 50257, 64), (2, 131072, 20), (1, 131075, 128), (1, 300001, 9),
         (200, 20003, 33), (5000, 40, 8), (1500, 600, 16), (2000, 2500, 100), (70, 9001, 31), (4, 1100000, 64)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", SIZES)
def test_rows(n, c, k, dt):
    x = _logits(n, c, dt, n * 31 + c)
    y = _labels(n, c, c)
    got = _run(x, y, k)
    _hold(x, y, got, k)
    again = _run(x, y, k)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits
    only = _run(x, None, 0)  # the entropy alone
    assert torch.equal(only[1], got[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("c", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 31, 40, 47, 63, 64, 65, 90, 100, 127, 128, 129])
@pytest.mark.parametrize("gap", [0, 3, 8])
def test_many_rows_of_few_classes(c, gap, dt):
    # a thread a row: rows that follow one another, rows on 16 bytes, others
    n = 20011
    wide = _logits(n, c + gap, dt, c)
    x = wide[:, :c]
    x[5], x[6, c // 2:], x[7] = -INF, -INF, 1.0
    if c > 2:
        x[8, 1:] = torch.finfo(DT[dt]).min
    y = _labels(n, c, c)
    for k in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):
        got = _run(x, y, k)
        _hold(x, y, got, k)
        if not k:
            got = got[:2]
        if k in (1, 8):
            m = n - 77
            part = _run(x, y, k, d_n=torch.tensor([m], dtype=torch.int32, device="cuda"))
            assert all(torch.equal(a[:m], b[:m]) for a, b in zip(part, got))
            assert all(bool((t[m:] == (77 if t.dtype == torch.int32 else 7)).all()) for t in part)
    z = x.clone() if gap == 0 else wide.clone()[:, :c]
    z[11, c - 1] = float("nan")
    z[12, 0] = INF
    bad = _run(z, y, 3)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[11:13] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(bad, _run(x, y, 3)))
    assert bool((bad[2][11:13] == -1).all()) and bool(torch.isnan(bad[3][11:13]).all()) and bool(torch.isnan(bad[1][11:13]).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", [(2500, 1300, 5), (2500, 2100, 32), (2500, 3001, 20), (2600, 5003, 100), (2600, 12001, 128), (2500, 16001, 40)])
@pytest.mark.parametrize("mask", [None, -1e9])
def test_many_rows_of_some_thousand_classes(n, c, k, mask, dt):
    # small CTAs that walk over their rows
    x = _logits(n, c, dt, c + k)
    if mask is not None:
        x[::3, k // 2:] = mask  # most classes of every third row are equal
        x[1::7, 3:] = -INF
    y = _labels(n, c, k)
    _hold(x, y, _run(x, y, k), k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vecs", [31, 32, 33, 64, 65, 128, 129, 256, 257, 384, 385, 512, 513, 768, 769, 1024, 1025, 1536, 1537,
                                  2048, 2049])
@pytest.mark.parametrize("start", [0, 3])
def test_rows_at_the_ends_of_the_forms(vecs, start, dt):
    # 1, 2 or 4 warps a row, as many vectors a lane as hold it; longer rows by blocks
    n, c = 21, vecs * (4 if dt == "f32" else 8)
    x = _logits(n, start + c + 1, dt, vecs)[:, start:start + c]
    x[3, 2:], x[4], x[5, : c // 2] = -INF, -INF, -INF
    x[6, c // 3:] = -7.0
    x[7, 1::2] = torch.finfo(DT[dt]).min
    y = _labels(n, c, c)
    for k in (1, 2, 24, 25, 32, 48, 49, 96, 97, 128):
        _hold(x, y, _run(x, y, k), k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,k", [(40, 100, 5), (40, 600, 20), (20, 3000, 64), (700, 5000, 20), (6, 40001, 64),
                                   (400, 20003, 100)])
@pytest.mark.parametrize("kept", [0, 1, 3, 50, "many"])
@pytest.mark.parametrize("mask", [-INF, -1e4, -1e9, "lowest"])
def test_masked_classes(n, c, k, dt, kept, mask):
    # (a finite mask leaves rows of which most classes are equal)
    x = _logits(n, c, dt, c + k)
    value = torch.finfo(DT[dt]).min if mask == "lowest" else mask
    off = torch.rand((n, c), generator=torch.Generator("cuda").manual_seed(c), device="cuda")
    if kept == "many":
        x[off < 0.5] = value
    else:
        x[off < torch.sort(off, dim=1, descending=True)[0][:, kept:kept + 1] if kept else off < 2] = value
    x[n // 2, : c // 2] = -INF
    y = _labels(n, c, k)
    _hold(x, y, _run(x, y, k), k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", [(3, 40), (30, 700), (5, 5000), (700, 5000), (400, 50257), (2, 131075)])
@pytest.mark.parametrize("k", [1, 20, 128])
def test_equal_logits(n, c, k, dt):
    # ties go to the lowest class: rows of one value, of -0 and 0, of two values, of few
    x = torch.zeros((n, c), device="cuda")
    g = torch.Generator("cuda").manual_seed(c)
    x[0] = 3.0
    x[1, ::2] = -0.0
    if n > 2:
        x[2] = torch.where(torch.rand(c, generator=g, device="cuda") < 0.3, 1.0, 2.0)
        x[2, : c // 2] = 1.0
        x[3 % n, c - 1] = 1.0
    if n > 4:
        x[4] = torch.randint(0, 12, (c,), generator=g, device="cuda").float()
        x[4, : c // 3] = 0.0
    x = x.to(DT[dt])
    y = _labels(n, c, 3)
    _hold(x, y, _run(x, y, k), k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", [(700, 60000), (3, 140000), (320, 20000)])
@pytest.mark.parametrize("k", [5, 20, 100])
def test_large_logits_in_a_few_lanes(n, c, k, dt):
    # all large logits at the same few lanes of a block: their maxima say little
    # about the k-th largest, and far more classes reach the bound than fit a list
    e = 4 if dt == "f32" else 8
    g = torch.Generator("cuda").manual_seed(k)
    x = torch.randn((n, c), generator=g, device="cuda") - 20
    lane = torch.arange(c, device="cuda") // e % 256
    for r in range(min(n, 8)):
        hot = (lane == 3) | (lane == 40 + r) | (lane == 200)
        x[r] = torch.where(hot, torch.rand(c, generator=g, device="cuda") * (1 + r), x[r])
    x[n - 1] = torch.where(lane == 100, torch.full_like(x[0], 4.0), x[n - 1])
    x = x.to(DT[dt])
    y = _labels(n, c, 5)
    _hold(x, y, _run(x, y, k), k)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("c", [20, 300, 2000, 9001, 131072])
def test_rows_at_any_level(c, dt):
    levels = torch.tensor([0.0, 1e3, -1e3, 1e5, -1e5, 1e9, -1e9, 1e30, -1e30, 3e38, -3e38], device="cuda")[:, None]
    g = torch.Generator("cuda").manual_seed(c)
    x = torch.randn((11, c), generator=g, device="cuda") * 3
    x = torch.where(levels == 0, x, levels + torch.where(levels.abs() > 1e6, x * levels.abs() * 2.0 ** -24, x)).to(DT[dt])
    x = torch.nan_to_num(x, posinf=3e38, neginf=-3e38)
    y = _labels(11, c, c).clamp(min=0)
    _hold(x, y, _run(x, y, 8), 8)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", [(30, 100), (30, 900), (6, 40000), (700, 9000)])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_nan_and_inf_stay_in_their_row(n, c, bad, dt):
    x = _logits(n, c, dt, c)
    y = _labels(n, c, 1)
    clean = _run(x, y, 6)
    hit = torch.arange(n, device="cuda") % 3 == 1
    x[hit, c - 1] = bad
    x[1, 0] = bad
    got = _run(x, y, 6)
    assert bool(torch.isnan(got[0][hit & (y >= 0)]).all()) and bool((got[0][hit & (y < 0)] == 0).all())
    assert bool(torch.isnan(got[1][hit]).all()) and bool((got[2][hit] == -1).all()) and bool(torch.isnan(got[3][hit]).all())
    assert all(torch.equal(a[~hit], b[~hit]) for a, b in zip(got, clean))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("c", [47, 128, 1001, 5001, 70000])
@pytest.mark.parametrize("start,gap", [(0, 0), (1, 3), (3, 8), (5, 1)])
def test_strides_and_rows_behind_the_count(c, start, gap, dt):
    n, m, k = 37, 21, 7
    wide = _logits(n, start + c + gap, dt, c)
    x = wide[:, start:start + c]
    y = _labels(n, c, 2)
    got = _run(x, y, k, d_n=torch.tensor([m], dtype=torch.int32, device="cuda"))
    _hold(x[:m], y[:m], [t[:m] for t in got], k)
    assert all(bool((t[m:] == (77 if t.dtype == torch.int32 else 7)).all()) for t in got)
    got = _run(x, y, k, d_n=torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert all(bool((t == (77 if t.dtype == torch.int32 else 7)).all()) for t in got)
    got = _run(x, y, k, d_n=torch.tensor([n + 5], dtype=torch.int32, device="cuda"))  # cut off at n
    _hold(x, y, got, k)


def test_labels_out_of_range_are_reported():
    for c in (40, 5000):
        x = _logits(8, c, "f32", 1)
        y = torch.tensor([0, 1, c, 3, -2, 5, -1, c - 1], dtype=torch.int32, device="cuda")
        logp, ent = torch.full((8,), 7.0, device="cuda"), torch.empty(8, device="cuda")
        sg.sg_logprobs(x, y, 8, None, logp, ent)
        with pytest.raises(sg.SgError) as e:
            sg.sg_stream_check()
        assert e.value.status == sg.SG_ERR_INVALID_INDEX
        y[2] = y[4] = -1
        want = _run(x, y, 0)
        assert torch.equal(logp, want[0]) and torch.equal(ent, want[1])


def test_offsets_past_32_bits():
    n, c = 33000, 70001
    x = torch.empty((n, c), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    y = _labels(n, c, 1)
    got = _run(x, y, 4)
    at = torch.tensor([0, 1, 17000, 30678, 30679, n - 1], device="cuda")
    _hold(x[at], y[at], [t[at] for t in got], 4)


def test_in_a_graph_and_on_other_streams():
    x = [_logits(64, c, "f32", c) for c in (100, 5000)]
    y = _labels(64, 100, 1)
    want = [_run(t, y, 10) for t in x]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t, o in zip(x, outs):
            sg.sg_logprobs(t, y, 64, None, *o)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for t, o in zip(x, outs):
            sg.sg_logprobs(t, y, 64, None, *o)
    for o in outs:
        for t in o:
            t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))


def test_two_streams_at_once():
    # a thread, a warp and four warps a row, blocks that walk over rows, a cluster a row
    cases = [(_logits(20000, 47, "f32", 1), 3), (_logits(3000, 900, "bf16", 2), 20), (_logits(500, 12000, "bf16", 3), 64),
             (_logits(400, 50257, "bf16", 4), 10), (_logits(3, 140000, "f32", 5), 100)]
    want = [_run(x, _labels(*x.shape, 6), k) for x, k in cases]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    streams = [torch.cuda.Stream() for _ in cases]
    labels = [_labels(*x.shape, 6) for x, _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for (x, k), y, o, s in zip(cases, labels, outs, streams):
            sg.sg_logprobs(x, y, len(x), None, *o, stream=s)
    torch.cuda.synchronize()
    sg.sg_stream_check()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("start,gap", [(1, 3), (3, 8), (0, 1)])
@pytest.mark.parametrize("vecs", [300, 600, 1200])
def test_register_rows_at_any_alignment(vecs, start, gap, dt):
    n, c, k = 37, vecs * (4 if dt == "f32" else 8) + 5, 30
    wide = torch.full((n, start + c + gap), float("nan"), dtype=DT[dt], device="cuda")
    wide[:, start:start + c] = _logits(n, c, dt, vecs)
    x, y, m = wide[:, start:start + c], _labels(n, c, 2), 30
    got = _run(x, y, k, d_n=torch.tensor([m], dtype=torch.int32, device="cuda"))
    _hold(x[:m], y[:m], [t[:m] for t in got], k)
    assert all(bool((t[m:] == (77 if t.dtype == torch.int32 else 7)).all()) for t in got)
