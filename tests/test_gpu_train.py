"""The training step (train.SageTrainer): its gradients against a dense
64-bit restatement on the sampled blocks, and that training learns."""
import numpy as np
import pytest
import torch

import synth
from sampling_gnn_mini_gb300 import binding as sg
from sampling_gnn_mini_gb300.train import SageTrainer, fit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _trainer(n=2000, dim=64, classes=7, fanouts=(6, 4), seeds=50, **kw):
    g = synth.chung_lu(n, 8.0, 2.1, 100.0, 0)
    return SageTrainer(sg.sg_graph_load(g.indptr.astype(np.int32), g.indices), dim, classes, list(fanouts), seeds, **kw)


def _reference(t, labels):
    """Loss, dW per layer and the table's gradient in 64 bits with autograd,
    on the blocks that the last forward() sampled."""
    H = t.H
    c = t.buf.counts.cpu().tolist()
    nodes = c[: H + 1]
    table = t.table.double().cpu().requires_grad_()
    W = [None] + [w.double().cpu().requires_grad_() for w in t.W[1:]]
    x = t.scale * table[t.buf.unique[: nodes[H]].long().cpu()]
    for h in range(H, 0, -1):
        ip = t.buf.indptr[h - 1][: nodes[h - 1] + 1].long().cpu()
        ix = t.buf.idx[h - 1][: int(ip[-1])].long().cpu()
        dst = torch.repeat_interleave(torch.arange(nodes[h - 1]), ip[1:] - ip[:-1])
        mean = torch.zeros(nodes[h - 1], x.shape[1], dtype=torch.float64).index_add(0, dst, x[ix])
        mean = mean / (ip[1:] - ip[:-1]).clamp(min=1)[:, None]
        y = torch.cat([x[: nodes[h - 1]], mean], 1) @ W[h].T
        x = torch.relu(y) if h > 1 else y
    loss = torch.nn.functional.cross_entropy(x[:, : t.n_classes], labels.long().cpu(), ignore_index=-1)
    loss.backward()
    return float(loss.detach()), [None] + [w.grad for w in W[1:]], table.grad


@pytest.mark.parametrize("fanouts,dim,classes", [((6, 4), 64, 7), ((5, 3, 2), 100, 128), ((8,), 32, 2)])
def test_gradients_match_autograd(fanouts, dim, classes):
    t = _trainer(dim=dim, classes=classes, fanouts=fanouts)
    rng = np.random.default_rng(dim)
    seeds = torch.from_numpy(rng.permutation(2000)[:50].astype(np.int32)).cuda()
    labels = torch.from_numpy(rng.integers(-1, classes, 50).astype(np.int32)).cuda()
    before = t.table.clone()
    logits = t.forward(seeds, 77)
    t.backward(labels, logits)
    sg.sg_stream_check()
    loss, dW, dT = _reference(t, labels)
    # tf32 operands (2^-11 each) through up to 3 layers forward and back, and
    # ReLU masks that differ where a pre-activation is that close to 0
    assert abs(float(t.total[0]) - loss) <= 5e-3 * abs(loss)
    for h in range(1, t.H + 1):
        d = (t.dW[h].double().cpu() - dW[h]).norm()
        assert float(d) <= 2e-2 * float(dW[h].norm()), h
    t.update()
    sg.sg_stream_check()
    got = (before - t.table).double().cpu() / t.lr_table
    assert float((got - dT).norm()) <= 2e-2 * float(dT.norm())
    untouched = dT.abs().sum(1) == 0
    used = torch.zeros(t.graph.n_nodes, dtype=torch.bool)
    used[t.buf.unique[: int(t.count(t.H))].long().cpu()] = True
    assert torch.equal(t.table.cpu()[~used], before.cpu()[~used])
    assert bool(untouched[~used].all())


def test_training_learns_and_repeats():
    # labels that the graph's neighbourhoods carry: a class per node, smoothed
    # once over sampled neighbours, is learnable through embeddings alone
    losses = []
    for _ in range(2):
        t = _trainer(n=600, dim=64, classes=5, fanouts=(5, 4), seeds=100, lr=0.05, lr_table=20.0)
        labels = (torch.arange(600, device="cuda") * 5 // 600).to(torch.int32)
        losses.append(fit(t, labels, 150, hash_seed=3))
        sg.sg_stream_check()
    assert losses[0] == losses[1]  # every sum has a fixed order
    assert 1.0 < losses[0][0] < 2.5
    assert np.mean(losses[0][-10:]) < 0.5 * losses[0][0]


def test_step_refuses_other_sizes():
    t = _trainer(seeds=10)
    with pytest.raises(ValueError):
        t.step(torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda"), 1)
    with pytest.raises(ValueError):
        _trainer(classes=129)
