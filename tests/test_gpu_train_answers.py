"""The training step with normalised hidden states and with a teacher: its
gradients against a dense 64-bit restatement on the sampled blocks; and the
answers that a trained model gives another one."""
import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_train import _trainer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


def _reference(t, labels, teacher, share, T):
    """Loss and gradients (W, norms, table) in 64 bits with autograd on the blocks
    that the last forward() sampled, and the logits."""
    H = t.H
    nodes = t.buf.counts.cpu().tolist()[: H + 1]
    table = t.table.double().cpu().requires_grad_()
    W = [None] + [w.double().cpu().requires_grad_() for w in t.W[1:]]
    N = {h: p.double().cpu().requires_grad_() for h, p in t.N.items()}
    x = t.scale * table[t.buf.unique[: nodes[H]].long().cpu()]
    for h in range(H, 0, -1):
        ip = t.buf.indptr[h - 1][: nodes[h - 1] + 1].long().cpu()
        ix = t.buf.idx[h - 1][: int(ip[-1])].long().cpu()
        dst = torch.repeat_interleave(torch.arange(nodes[h - 1]), ip[1:] - ip[:-1])
        mean = torch.zeros(nodes[h - 1], x.shape[1], dtype=torch.float64).index_add(0, dst, x[ix])
        mean = mean / (ip[1:] - ip[:-1]).clamp(min=1)[:, None]
        x = torch.cat([x[: nodes[h - 1]], mean], 1) @ W[h].T
        if h > 1:
            x = torch.relu(x)
            if h - 1 in N:
                x = torch.nn.functional.layer_norm(x, (128,), N[h - 1][0], N[h - 1][1], 1e-5)
    x = x[:, : t.n_classes]
    loss = torch.nn.functional.cross_entropy(x, labels.long().cpu(), ignore_index=-1)
    if teacher is not None:
        ids, v = teacher[0].long().cpu(), teacher[1].double().cpu()
        q = torch.softmax(torch.where(ids >= 0, v, -float("inf")) / T, 1)
        logp = torch.log_softmax(x / T, 1).gather(1, ids.clamp(min=0))
        loss = (1 - share) * loss + share * T * T * torch.where(q > 0, q * (torch.log(q) - logp), 0.0).sum(1).mean()
    loss.backward()
    return float(loss.detach()), [None] + [w.grad for w in W[1:]], {h: p.grad for h, p in N.items()}, table.grad, x.detach()


@pytest.mark.parametrize("fanouts,classes,norm,taught", [((6, 4), 7, True, False), ((6, 4), 100, False, True),
                                                         ((5, 3, 2), 128, True, True), ((8,), 12, True, True)])
def test_gradients_match_autograd(fanouts, classes, norm, taught):
    t = _trainer(classes=classes, fanouts=fanouts, norm=norm)
    rng = np.random.default_rng(classes)
    seeds = torch.from_numpy(rng.permutation(2000)[:50].astype(np.int32)).cuda()
    labels = torch.from_numpy(rng.integers(-1, classes, 50).astype(np.int32)).cuda()
    teacher = None
    for h in t.N:
        t.N[h] += 0.1 * torch.randn(2, 128, generator=torch.Generator("cuda").manual_seed(h), device="cuda")
    if taught:
        teacher = _trainer(classes=classes, fanouts=fanouts, seed=5).predict(seeds, 3, k=min(16, classes))[:2]
    before = t.table.clone()
    logits = t.forward(seeds, 77)
    t.backward(labels, logits, teacher, 0.3, 2.0)
    sg.sg_stream_check()
    loss, dW, dN, dT, _ = _reference(t, labels, teacher, 0.3, 2.0)
    # tf32 operands (2^-11 each) through up to 3 layers forward and back, and
    # ReLU masks that differ where a pre-activation is that close to 0
    assert abs(float(t.total[0]) - loss) <= 5e-3 * abs(loss)
    for h in range(1, t.H + 1):
        assert float((t.dW[h].double().cpu() - dW[h]).norm()) <= 2e-2 * float(dW[h].norm()), h
    for h in dN:
        for p in (0, 1):
            assert float((t.dN[h][p].double().cpu() - dN[h][p]).norm()) <= 2e-2 * float(dN[h][p].norm()), (h, p)
    norms = {h: p.clone() for h, p in t.N.items()}
    t.update()
    sg.sg_stream_check()
    got = (before - t.table).double().cpu() / t.lr_table
    assert float((got - dT).norm()) <= 2e-2 * float(dT.norm())
    for h in norms:
        assert torch.equal(t.N[h], torch.add(norms[h], t.dN[h], alpha=-t.lr_norm))


def test_answers_of_the_model():
    t = _trainer(classes=20, norm=True)
    seeds = torch.randperm(2000, device="cuda", generator=torch.Generator("cuda").manual_seed(1))[:50].int()
    labels = (seeds % 21 - 1).int()
    ids, logps, entropy, logp = t.predict(seeds, 9, k=25, labels=labels)
    sg.sg_stream_check()
    all_logp = torch.log_softmax(t.Y[1][:50, :20].double(), 1)
    v, order = torch.sort(all_logp, dim=1, descending=True, stable=True)
    assert torch.equal(ids[:, :20].long(), order) and bool((ids[:, 20:] == -1).all())
    assert float((logps[:, :20].double() - v).abs().max()) <= 1e-5 and bool((logps[:, 20:] == -float("inf")).all())
    assert float((entropy.double() + (all_logp.exp() * all_logp).sum(1)).abs().max()) <= 1e-5
    want = torch.where(labels < 0, 0.0, all_logp.gather(1, labels.clamp(min=0).long()[:, None])[:, 0])
    assert float((logp.double() - want).abs().max()) <= 1e-5
    with pytest.raises(ValueError):
        t.predict(seeds[:3], 9)


def test_steps_with_a_teacher_repeat():
    # the same bits from the same start: every sum has a fixed order
    runs = []
    for _ in range(2):
        big, small = _trainer(classes=9, norm=True, seed=4), _trainer(classes=9, norm=True, seeds=50)
        seen = []
        for k in range(5):
            seeds = torch.randperm(2000, device="cuda", generator=torch.Generator("cuda").manual_seed(k))[:50].int()
            labels = (seeds % 9).int()
            seen.append(small.step(seeds, labels, k, teacher=big.predict(seeds, k, k=4)[:2]).clone())
            big.step(seeds, labels, k)
        sg.sg_stream_check()
        runs.append((torch.stack(seen), small.table.clone(), small.N[1].clone(), big.W[1].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*runs)) and bool(torch.isfinite(runs[0][0]).all())
    with pytest.raises(ValueError):
        small.step(seeds, labels, 1, teacher=big.predict(seeds, 1)[:2], share=1.5)
