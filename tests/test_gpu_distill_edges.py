"""Values and logits of sg_distill at the ends of what its description allows."""
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_distill import DT, INF, _case, _reference, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


@pytest.mark.parametrize("n,c", [(20, 60), (300, 900), (6, 40001), (700, 9001)])
@pytest.mark.parametrize("T", [2.0, 30.0])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_bad_values_of_classes_without_a_logit(n, c, T, bad):
    # a value that is NaN or +inf makes its row's loss NaN, also where every entry's logit is -inf
    x, ids, v = _case(n, c, 5, "f32", c)
    ids = ids.clamp(min=0)
    v = torch.nan_to_num(v, neginf=0.0)
    clean = _run(x, ids, v, T, mean=False)
    v[1, 0] = bad
    x[1].scatter_(0, ids[1].long(), -INF)
    got = _run(x, ids, v, T, mean=False)
    keep = torch.arange(n, device="cuda") != 1
    assert bool(torch.isnan(got[0][1])) and bool(torch.isnan(got[1][0]))
    assert bool(torch.isnan(got[2][1].gather(0, ids[1].long())).all())
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[2][keep], clean[2][keep])
    # and +inf where the values are good
    v[1, 0] = 1.0
    assert float(_run(x, ids, v, T, mean=False)[0][1]) == INF


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,c", [(20, 60), (300, 900), (6, 40001), (700, 9001)])
@pytest.mark.parametrize("T", [0.001, 0.1, 0.7, 1.0])
def test_a_teachers_class_at_the_types_lowest_value(n, c, T, dt):
    # the loss is T q times the logits' difference, which T below 1 leaves in range
    x, ids, v = _case(n, c, 5, dt, c)
    ids = ids.clamp(min=0)
    v = torch.nan_to_num(v, neginf=0.0) * T  # q does not fall below the type's range
    x[1, ids[1, 1].long()] = torch.finfo(DT[dt]).min
    x[0, ids[0].long()] = torch.finfo(DT[dt]).min
    got = _run(x, ids, v, T, mean=False)
    want, tol = _reference(x, ids, v, T, False, 1.0)[:2]
    fits = want < 3.4e38  # (T = 1: q just below 1 may not)
    assert bool(fits[1]) and bool((((got[0].double() - want).abs() <= tol) | ~fits).all())
    assert bool(torch.isfinite(got[0][fits]).all()) and bool(torch.isfinite(got[2]).all())
