"""How exact the orthogonalisation's products are, and the ends of its range
(sg_orthogonalise, sg_muon_step), against 64 bits.

Operands are pairs of fp16 terms of 256 times the value: off by d = 2^-22 of an
entry (or by 2^-25 of 256 times it, where the second term is below fp16's
normal range).  With ONE term, or a cross product left out, they are off by 2^-12 or
so, which the limits here do not let pass.

Five steps.  A step's error relative to singular values near 1 is at most |f'(t)| <= 4
times d for X's rounding, (|b| + 2 |c| t^2) t^3 < 15 d for A's and some 5 d for B's:
24 d; the step before it counts up to 4 times, earlier ones are made of small
singular values, whose relative error does not grow.  That is 150 d if all roundings
were as large as they can be and alike in sign; uniform ones have 0.4 of that: 60 d =
1.4e-5.  Limit: 2e-5 of the Frobenius norm.

One step.  a alone gives X itself: its rounding (d, and that of the norm and the
scaling, as much again).  b alone gives A X: three roundings of X, one of A, one of B
and two sums, which the tensor core cuts by up to 2^-24 at each of 8 accumulations:
limit 32 d.  All three, with A A X: limit 64 d.  (c alone is not held to a limit: the
entries of c A A, about 1 / m^2, would have only their distance to the least step
2^-25 / 256, which is small beside a I.)"""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg

pytestmark = pytest.mark.gpu
D = 2.0 ** -22
COEF = (3.4445, -4.7750, 2.0315)
# one launch with 256, 64 and 128 columns a CTA (upright and tall); launches of
# products with tiles of 64, 128 and 256 columns
SHAPES = [(128, 200), (100, 256), (128, 512), (128, 1000), (128, 2048), (200, 128), (1900, 120), (1001, 603), (130, 513),
          (256, 2049), (512, 4096), (1024, 4096)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _reference(u, coef, eps=1e-7):
    x = u.double()
    x = x / (x.norm() + np.float64(np.float32(eps)))
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for step in coef:
        a, b, c = (np.float64(np.float32(v)) for v in step)
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.T if tall else x


def _ws(count, rows, cols):
    ws = sg.aligned_workspace(sg.sg_orthogonalise_workspace(count, rows, cols))
    ws.fill_(0xEE)
    return ws


def _run(g, **kw):
    k = g.shape[0] if g.dim() == 3 else 1
    out = torch.full_like(g, 7.0)
    sg.sg_orthogonalise(g, out, _ws(k, g.shape[-2], g.shape[-1]), **kw)
    sg.sg_stream_check()
    return out


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_five_steps_are_as_exact_as_the_pairs(rows, cols):
    g = torch.randn((rows, cols), generator=_gen(rows + cols), device="cuda")
    assert _off(_run(g), _reference(g, [COEF] * 5)) <= 2e-5


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_each_product_alone(rows, cols):
    g = torch.randn((rows, cols), generator=_gen(rows * cols), device="cuda")
    flat = 2.0 ** -25 / 256 * np.sqrt(rows * cols)  # of the norm: every entry off by the least step
    for coef, limit in (((1.0, 0.0, 0.0), 2 * D + flat), ((0.0, 1.0, 0.0), 32 * D), (COEF, 64 * D)):
        got = _run(g, steps=1, coef=[coef])
        assert _off(got, _reference(g, [coef])) <= limit, coef


@pytest.mark.parametrize("rows,cols", [(128, 200), (128, 2048), (200, 128), (260, 333), (512, 4096)])
def test_a_weight_step_is_as_exact(rows, cols):
    gen = _gen(rows - cols)
    w = torch.zeros((rows, cols), device="cuda")  # the step alone is seen
    g, m = (torch.randn((rows, cols), generator=gen, device="cuda") * 1e-3 for _ in range(2))
    w2, m2 = torch.empty_like(w), torch.empty_like(m)
    sg.sg_muon_step(w, g, m, w2, m2, _ws(1, rows, cols), lr=1.0, momentum=0.5)
    sg.sg_stream_check()
    u = g.double() + 0.5 * (0.5 * m.double() + g.double())
    assert _off(w2, -_reference(u, [COEF] * 5)) <= 2e-5


@pytest.mark.parametrize("rows,cols", [(128, 200), (60, 1000), (128, 2048), (300, 100), (300, 280), (140, 3000)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nan_and_inf_stay_in_their_matrix(rows, cols, bad):
    # one entry that is not finite: nothing is left of its matrix, the others keep their bits
    g = torch.randn((3, rows, cols), generator=_gen(rows), device="cuda") * 1e-3
    clean = _run(g)
    g[1, rows // 2, cols // 3] = bad
    out = _run(g)
    assert bool(torch.isnan(out[1]).all())
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    w = torch.randn((3, rows, cols), generator=_gen(cols), device="cuda")
    m = torch.zeros_like(g)
    w2, m2 = torch.empty_like(w), torch.empty_like(m)
    sg.sg_muon_step(w, g, m, w2, m2, _ws(3, rows, cols), lr=0.1)
    sg.sg_stream_check()
    assert bool(torch.isnan(w2[1]).all()) and bool(torch.isfinite(w2[[0, 2]]).all())
    assert torch.equal(torch.isfinite(m2), torch.isfinite(g))


@pytest.mark.parametrize("rows,cols", [(1, 65536), (65536, 5), (130, 65536), (65536, 129)])
def test_the_longest_sides(rows, cols):
    g = torch.randn((rows, cols), generator=_gen(rows), device="cuda")
    assert _off(_run(g), _reference(g, [COEF] * 5)) <= 2e-5


def test_the_largest_square():
    g = torch.randn((8192, 8200), generator=_gen(1), device="cuda")
    assert _off(_run(g, steps=1), _reference(g, [COEF])) <= 2e-5


def test_past_31_bit_offsets():
    # 2.4e9 elements.  The last matrices' results are those of the same matrices
    # alone.  Rows that do not overlap, so A is diagonal: with s_i = |x_i|^2 row
    # i becomes (a + b s_i + c s_i^2) x_i, up to the bf16 rounding of the output
    count, rows, cols, per = 9, 4096, 65536, 16
    gen = _gen(2)
    v = torch.randn((count, rows, per), generator=gen, device="cuda").bfloat16()
    v *= (1 + torch.arange(rows, device="cuda") % 7)[None, :, None]
    g = torch.zeros((count, rows, cols), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(rows, device="cuda")[:, None] * per + torch.arange(per, device="cuda")
    for q in range(count):
        g[q].scatter_(1, at, v[q])
    coef = (1.0, -300.0, 20000.0)
    alone = [_run(g[q], steps=1, coef=[coef]) for q in (0, 7, 8)]
    ws = sg.aligned_workspace(sg.sg_orthogonalise_workspace(count, rows, cols))
    sg.sg_orthogonalise(g, g, ws, steps=1, coef=[coef])
    sg.sg_stream_check()
    for q, want in zip((0, 7, 8), alone):
        assert torch.equal(g[q], want)
    for q in range(count):
        x = v[q].double()
        x = x / (x.norm() + 1e-7)
        s = x.square().sum(1, keepdim=True)
        got = g[q].gather(1, at).double()
        assert _off(got, (coef[0] + coef[1] * s + coef[2] * s * s) * x) <= 2.0 ** -8 + 2e-5
        g[q].scatter_(1, at, torch.zeros_like(v[q]))
        assert not bool(g[q].any())
