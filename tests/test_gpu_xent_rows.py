"""Softmax cross-entropy (sg_xent): rows that meet one another in a kernel, and
rows of unusual logits, in every form of the kernel.

The forms, by the rows' length and number (fp32): a cluster of 1 to 8 CTAs a row
for few rows, and clusters that walk over their rows, `step` rows apart, for
many."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_xent import _check, _ws

pytestmark = pytest.mark.gpu


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
