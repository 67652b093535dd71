"""Softmax cross-entropy (sg_xent): rows that meet one another in a kernel, and
rows of unusual logits, in every form of the kernel.

The forms, by the rows' length and number (fp32): a thread a row, warps (in one
cluster or many blocks), a cluster of 1 to 8 CTAs a row for few rows, and
clusters that walk over their rows, `step` rows apart, for many.

Tolerances (u = 2^-24, d = m - x): a logit's difference to the row's (or a warp's)
largest is rounded once and scaled once, and the base-2 exponential is off by
2^-22, so an exponential is off by (8 + 2 d) u relative, and 8 u more where a
warp's sum is brought to the row's maximum.  With the sum of C terms the sum of
exponentials is off by (2 E[d] + C / 256 + 48) u, E[d] the mean of d under the
softmax.  The loss is off by that, by 2 u of its two parts m - x_label and log z,
and by 8 u of the logarithm; none of it grows with the row's level.  The
gradient is off by w (p (64 + 4 d + C / 256 + 2 E[d]) + 2) u; a bf16 gradient has to be
the rounding of a value within that."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_xent import _check, _ws

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _run(x, labels, mean=True, grad=True):
    """(loss, total, gradient) of sg_xent; labels: numpy int32."""
    n, c = x.shape
    loss, total = torch.full((n,), 7.0, device="cuda"), torch.full((2,), 7.0, device="cuda")
    g = torch.full_like(x, 7.0) if grad else None
    sg.sg_xent(x, torch.from_numpy(labels).cuda(), n, None, loss, total, g, _ws(n, c), mean=mean)
    sg.sg_stream_check()
    return loss, total, g


# classes (fp32), threads and CTAs of a cluster that streams such rows
STREAMED = [(2500, 256, 1), (9001, 512, 1), (20003, 512, 2), (40001, 512, 4), (60001, 512, 8)]


@pytest.mark.parametrize("ignored", [1, 3])
@pytest.mark.parametrize("c,threads,ctas", STREAMED)
def test_ignored_rows_between_used_ones(c, threads, ctas, ignored):
    # a cluster's used rows with 1 or 3 ignored ones between them, at levels so
    # far apart (0, 8) that one row's statistics would show in another's result
    step = torch.cuda.get_device_properties(0).multi_processor_count * (1024 // threads) // ctas
    n = 9 * step + step // 3
    gen = torch.Generator(device="cuda")
    gen.manual_seed(c + ignored)
    turn = np.arange(n) // step
    x = torch.randn((n, c), generator=gen, device="cuda")
    x += torch.from_numpy((turn // (ignored + 1) % 2 * 8.0).astype(np.float32)).cuda()[:, None]
    labels = np.random.default_rng(c).integers(0, c, n).astype(np.int32)
    labels[turn % (ignored + 1) != 0] = -1
    x[torch.from_numpy(labels == -1).cuda()] = float("nan")  # not looked at
    loss, total, grad = _run(x, labels)
    first = (loss.clone(), total.clone(), grad.clone())
    _check(x.nan_to_num(0.0), labels, loss, total, grad, True, 1.0)
    for _ in range(4):
        again = _run(x, labels)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    # the loss alone takes no time for the gradient between the rows
    only = _run(x, labels, grad=False)
    assert torch.equal(only[0], first[0]) and torch.equal(only[1], first[1])


# ------------------------------------------------------- rows of any level
# rows and classes of every form (fp32; bf16 rows take a form of half the length)
FORMS = [(300, 10), (8, 40), (9, 1000), (300, 130), (270, 1000), (8, 1100), (8, 2500), (8, 5000), (8, 9001), (8, 70001),
         (8, 140001), (1000, 2500), (480, 9001), (240, 20003), (240, 40001), (130, 60001)]
LEVELS = [0.0, 1e3, -1e3, 1e4, -1e4, 6e4, -6e4, 1e6, -1e6, 1e9, -1e9, 1e10, -1e10, 1e30, -1e30, 3e38]


def _rounded(x):
    """float64 values rounded to 8 bits of significand, ties to even (bfloat16
    in its normal range)."""
    bits = x.contiguous().view(torch.int64)
    bits = bits + ((1 << 44) - 1) + ((bits >> 45) & 1)
    return (bits & ~((1 << 45) - 1)).view(torch.float64)


def _hold(x, labels, loss, grad):
    """Every row of the mean loss and its gradient against 64 bits."""
    n, c = x.shape
    x64, y = x.double(), torch.from_numpy(labels).cuda().long()
    assert bool((y >= 0).all())
    m = x64.amax(1, keepdim=True)
    d = m - x64
    e = torch.exp(-d)
    z = e.sum(1, keepdim=True)
    p = e / z
    mean_d = torch.where(p > 0, p * d, torch.zeros_like(d)).sum(1)
    dy = d.gather(1, y[:, None])[:, 0]
    want, lerr = torch.log(z)[:, 0] + dy, U * (2 * dy + 2 * torch.log(z)[:, 0] + 2 * mean_d + c / 256 + 64)
    off = (loss.double() - want).abs()
    # (a difference of two logits may pass the largest fp32 number)
    assert bool(((off <= lerr) | ((want > 3.4e38) & (loss > 3.4e38))).all()), (off / lerr).max()
    w = 1.0 / n
    g = w * p
    g.scatter_add_(1, y[:, None], torch.full_like(z, -w))
    tol = w * (torch.where(p > 0, p * (64 + 4 * d + c / 256 + 2 * mean_d[:, None]), torch.zeros_like(d)) + 2) * U
    got = grad.double()
    if grad.dtype == torch.bfloat16:
        assert bool(((_rounded(g - tol) <= got) & (got <= _rounded(g + tol))).all())
    else:
        assert bool(((got - g).abs() <= tol).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", FORMS)
@pytest.mark.parametrize("equal", [True, False])
def test_rows_at_any_level(n, c, dt, equal):
    # rows of equal logits and rows with a spread (as far as the type has
    # neighbours there): the loss does not depend on the level
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n + c)
    level = torch.tensor(LEVELS, device="cuda")[torch.arange(n, device="cuda") % len(LEVELS)][:, None]
    x = torch.randn((n, c), generator=gen, device="cuda") * (0.0 if equal else 3.0)
    x = torch.where(level == 0, x, level + torch.where(level.abs() > 1e7, x * level.abs() * 2.0 ** -24, x)).to(DT[dt])
    x = torch.nan_to_num(x, posinf=3e38)
    labels = np.random.default_rng(c).integers(0, c, n).astype(np.int32)
    loss, total, grad = _run(x, labels)
    _hold(x, labels, loss, grad)
    assert not bool(torch.isnan(total).any())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", FORMS)
@pytest.mark.parametrize("kept", [8, 64, None])
def test_classes_masked_by_a_large_value(n, c, dt, kept):
    # whole warps and CTAs hold nothing but a finite mask value; None: one
    # warp's vectors of a row of 1,100 fp32 classes and more
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n * c)
    x = 2 * torch.randn((n, c), generator=gen, device="cuda")
    masks = torch.tensor([-1e4, -1e6, -1e9, -1e10, -1e20, -1e30, -1e36, -3e38], device="cuda")
    value = masks[torch.arange(n, device="cuda") % len(masks)][:, None]
    at = torch.arange(c, device="cuda")
    off = (at >= 896) & (at < 1024) if kept is None else at >= kept
    x = torch.where(off[None, :], value.expand(n, c), x).to(DT[dt])
    rng = np.random.default_rng(c)
    labels = rng.integers(0, min(c, 896 if kept is None else kept), n).astype(np.int32)
    loss, total, grad = _run(x, labels)
    _hold(x, labels, loss, grad)
    assert bool(torch.isfinite(total).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", FORMS)
def test_sure_rows(n, c, dt):
    # one class far above the others, and it is the label (or the next one is)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n + 3 * c)
    top = torch.tensor([12.0, 16.0, 30.0, 1e2, 1e3, 1e5, 1e9], device="cuda")[torch.arange(n, device="cuda") % 7]
    at = torch.randint(0, c, (n,), generator=gen, device="cuda")
    x = torch.zeros((n, c), device="cuda").scatter_(1, at[:, None], top[:, None]).to(DT[dt])
    for shift in (0, 1):
        labels = ((at + shift) % c).int().cpu().numpy()
        loss, _, grad = _run(x, labels)
        _hold(x, labels, loss, grad)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_reaches_the_masked_classes_of_its_row(n, c, dt, bad):
    # all classes but a few masked with -inf: whole warps have nothing to add,
    # and their part of a row's gradient is NaN all the same; other rows keep theirs
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n + 5 * c)
    x = torch.randn((n, c), generator=gen, device="cuda")
    x[:, 8:] = float("-inf")
    x = x.to(DT[dt])
    labels = np.random.default_rng(c).integers(0, min(c, 8), n).astype(np.int32)
    hit = torch.arange(n, device="cuda") % 3 == 1
    clean = _run(x, labels)
    _hold(x, labels, clean[0], clean[2])
    x[hit, 5] = bad
    loss, total, grad = _run(x, labels)
    assert bool(torch.isnan(loss[hit]).all()) and bool(torch.isnan(grad[hit]).all()) and bool(torch.isnan(total[0]))
    assert torch.equal(loss[~hit], clean[0][~hit]) and torch.equal(grad[~hit], clean[2][~hit])


@pytest.mark.parametrize("n,c", FORMS)
def test_small_losses(n, c):
    # two classes left of each row, d apart, the label the upper one: the sum is
    # 1 + e, e = exp(-d), with one rounding (u) and e's own (8 + 2 d relative,
    # 8 more where it comes from another warp); the logarithm is within an ulp
    # of its value; the loss is never below 0
    rng = np.random.default_rng(n + c)
    for turn in range(max(1, 200 // n)):
        d = np.exp(rng.uniform(np.log(1.0), np.log(16.0), n)).astype(np.float32)
        top = rng.integers(0, c, n)
        other = (top + 1 + rng.integers(0, c - 1, n)) % c
        level = rng.integers(-4, 5, n).astype(np.float32) * 4  # so that level - d is rounded at most by 2^-20
        x = torch.full((n, c), float("-inf"), device="cuda")
        row = torch.arange(n, device="cuda")
        x[row, torch.from_numpy(top).cuda()] = torch.from_numpy(level).cuda()
        x[row, torch.from_numpy(other).cuda()] = torch.from_numpy(level - d).cuda()
        gap = level.astype(np.float64) - (level - d).astype(np.float64)
        loss, _, _ = _run(x, top.astype(np.int32))
        e = np.exp(-gap)
        want, got = np.log1p(e), loss.double().cpu().numpy()
        assert np.all(got >= 0)
        assert np.all(np.abs(got - want) <= U * (1 + e * (16 + 2 * gap) + 2 * want))
