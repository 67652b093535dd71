"""A training loop's step on sampled mini-batches, through the C ABI: learned
node embeddings under GraphSAGE-mean layers, a softmax loss over the seeds,
and the updates.

Per step (V_h, block h: the sampler's node lists and blocks, Fig. 1 of the
GARDEN page; H hops, hidden width 128):
  1. sg_sampler_run, sg_transpose_blocks
  2. sg_embed_fwd     X_H = scale * table[V_H]
  3. h = H .. 1:      M_h = sg_aggregate_fwd(block h, X_h);
                      Y_h = [X_h | M_h] W_h^T, X_{h-1} = ReLU(Y_h)  (sg_sage_fwd)
  4. sg_xent          on the first n_classes columns of Y_1 (no ReLU after the
                      last layer): the seeds' loss and its gradient
  5. h = 1 .. H:      dW_h, dX (own rows), dM_h  (sg_sage_bwd); the gradient of
                      X_h = the transpose of block h on dM_h (sg_aggregate_bwd_t)
                      plus dX on the first |V_{h-1}| rows
  6. sg_muon_step     each W_h;  sg_embed_bwd (SG_GRAD_ADD) the table's rows,
                      a sparse SGD step
Sizes that depend on the sample stay on the device; a step does not
synchronise.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import binding as sg

HIDDEN = 128  # output width of sg_sage_fwd


class SageTrainer:
    """Learns a table of n_nodes x dim embeddings and the weights of
    len(fanouts) GraphSAGE layers for the classification of nodes into at most
    128 classes."""

    def __init__(self, graph: sg.Graph, dim: int, n_classes: int, fanouts: Sequence[int], n_seeds: int,
                 lr: float = 0.02, lr_table: float = 1.0, momentum: float = 0.95, scale: float = 1.0, seed: int = 0,
                 device="cuda"):
        if not 1 <= n_classes <= HIDDEN:
            raise ValueError("SageTrainer: 1 to %d classes" % HIDDEN)
        if n_seeds < 1:
            raise ValueError("SageTrainer: at least one seed")
        self.graph, self.n_classes, self.n_seeds = graph, int(n_classes), int(n_seeds)
        self.fanouts = [int(f) for f in fanouts]
        self.lr, self.lr_table, self.momentum = lr, lr_table, momentum
        # of the looked-up rows, which start with unit norm; it multiplies the
        # gradient as well, so a step moves the rows in use by lr_table * scale^2
        self.scale = float(scale)
        H = self.H = len(self.fanouts)
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def randn(*shape, std):
            return torch.empty(shape, device=device).normal_(0, std, generator=gen)
        self.table = randn(graph.n_nodes, dim, std=1 / (self.scale * math.sqrt(dim)))
        self.dims = [HIDDEN] * H + [dim]  # width of X_h, h = 0 .. H
        self.W = [None] + [randn(HIDDEN, 2 * self.dims[h], std=1 / math.sqrt(2 * self.dims[h])) for h in range(1, H + 1)]
        self.m = [None] + [torch.zeros_like(w) for w in self.W[1:]]

        self.bounds = sg.sg_sampler_bounds(graph, n_seeds, self.fanouts)
        self.buf = sg.SampleBuffers(self.bounds, device, graph, n_seeds, self.fanouts)
        self.tbuf = sg.TransposedBuffers(self.bounds, device)
        nb = self.nb = self.bounds.max_nodes
        self.d_seed = torch.zeros(1, dtype=torch.int64, device=device)

        def rows(h, width):
            return torch.empty((nb[h], width), device=device)
        self.X = [rows(h, self.dims[h]) for h in range(H + 1)]
        self.M = [None] + [rows(h - 1, self.dims[h]) for h in range(1, H + 1)]
        self.Y = [None] + [rows(h - 1, HIDDEN) for h in range(1, H + 1)]
        self.dW = [None] + [torch.empty_like(w) for w in self.W[1:]]
        # G[h]: gradient of X_h (of Y_1 for h = 0: columns past n_classes stay zero)
        self.G = [torch.zeros((nb[0], HIDDEN), device=device)] + [rows(h, self.dims[h]) for h in range(1, H + 1)]
        self.dX = [None] + [rows(h - 1, self.dims[h]) for h in range(1, H + 1)]
        self.dM = [None] + [rows(h - 1, self.dims[h]) for h in range(1, H + 1)]
        self.ones = torch.ones((nb[0], HIDDEN), device=device)  # "pre-activation" of the last layer: nothing is masked
        self.loss = torch.empty(n_seeds, device=device)
        self.total = torch.zeros(2, device=device)
        self.ws_xent = sg.aligned_workspace(sg.sg_xent_workspace(n_seeds, self.n_classes), device)
        self.ws_sage = sg.aligned_workspace(max(sg.sg_sage_bwd_workspace(nb[h - 1], self.dims[h], sg.SG_F32)
                                                for h in range(1, H + 1)), device)
        self.ws_muon = sg.aligned_workspace(max(sg.sg_orthogonalise_workspace(1, HIDDEN, 2 * self.dims[h])
                                                for h in range(1, H + 1)), device)
        self.ws_embed = sg.aligned_workspace(sg.sg_embed_bwd_workspace(nb[H], graph.n_nodes, dim, sg.SG_GRAD_ADD), device)

    def count(self, h: int) -> torch.Tensor:
        """|V_h| on the device."""
        return self.buf.counts[h:h + 1]

    def forward(self, seeds: torch.Tensor, hash_seed: int) -> torch.Tensor:
        """Samples and runs the layers; returns the seeds' logits."""
        H, nb = self.H, self.nb
        self.d_seed.fill_(hash_seed if hash_seed < (1 << 63) else hash_seed - (1 << 64))
        sg.sg_sampler_run(self.graph, seeds, self.fanouts, 0, self.buf, d_seed=self.d_seed)
        sg.sg_embed_fwd(self.table, self.buf.unique, nb[H], self.count(H), self.scale, self.X[H])
        for h in range(H, 0, -1):
            sg.sg_aggregate_fwd(self.buf.indptr[h - 1], self.buf.idx[h - 1], nb[h - 1], nb[h], self.buf.dims(h),
                                self.X[h], self.M[h])
            sg.sg_sage_fwd(self.X[h], self.M[h], self.W[h], nb[h - 1], self.count(h - 1), self.X[h - 1], self.Y[h])
        return self.Y[1][: self.n_seeds, : self.n_classes]

    def backward(self, labels: torch.Tensor, logits: torch.Tensor) -> None:
        """The loss and every gradient of the batch that forward() ran."""
        H, nb = self.H, self.nb
        sg.sg_xent(logits, labels, self.n_seeds, None, self.loss, self.total,
                   self.G[0][: self.n_seeds, : self.n_classes], self.ws_xent)
        sg.sg_transpose_blocks(self.buf, self.tbuf)
        t = self.tbuf
        for h in range(1, H + 1):
            self.dX[h].zero_()  # rows past |V_{h-1}| are added below as well
            sg.sg_sage_bwd(self.X[h], self.M[h], self.W[h], nb[h - 1], self.count(h - 1),
                           self.ones if h == 1 else self.Y[h], self.G[h - 1], self.dW[h], self.dX[h], self.dM[h],
                           self.ws_sage)
            sg.sg_aggregate_bwd_t(t.tptr[h - 1], t.tdst[h - 1], t.tw[h - 1], nb[h], nb[h - 1], self.buf.dims(h),
                                  self.dM[h], self.G[h])
            self.G[h][: nb[h - 1]] += self.dX[h]

    def update(self) -> None:
        """Muon on the weights, sparse SGD on the table's rows of the batch."""
        H = self.H
        for h in range(1, H + 1):
            r, c = self.W[h].shape
            sg.sg_muon_step(self.W[h], self.dW[h], self.m[h], self.W[h], self.m[h], self.ws_muon, lr=self.lr,
                            momentum=self.momentum, scale=math.sqrt(max(1.0, r / c)))
        sg.sg_embed_bwd(self.buf.unique, self.nb[H], self.count(H), self.graph.n_nodes, self.G[H],
                        -self.lr_table * self.scale, self.table, sg.SG_GRAD_ADD, self.ws_embed)

    def step(self, seeds: torch.Tensor, labels: torch.Tensor, hash_seed: int) -> torch.Tensor:
        """One training step on n_seeds distinct seeds (device int32) with
        their labels (-1: none); returns {mean loss, labelled seeds} on the
        device."""
        if seeds.numel() != self.n_seeds or labels.numel() != self.n_seeds:
            raise ValueError("SageTrainer.step: expected %d seeds and labels" % self.n_seeds)
        logits = self.forward(seeds, hash_seed)
        self.backward(labels, logits)
        self.update()
        return self.total


def fit(trainer: SageTrainer, labels: torch.Tensor, steps: int, hash_seed: int = 0,
        nodes: Optional[torch.Tensor] = None) -> list:
    """Trains on random batches of `nodes` (all of them when None) with
    labels[node]; returns the mean loss of every step (read at the end)."""
    dev = labels.device
    pool = torch.arange(trainer.graph.n_nodes, device=dev, dtype=torch.int32) if nodes is None else nodes
    gen = torch.Generator(device=dev)
    gen.manual_seed(hash_seed)
    seen = []
    for k in range(steps):
        seeds = pool[torch.randperm(len(pool), device=dev, generator=gen)[: trainer.n_seeds]]
        seen.append(trainer.step(seeds, labels[seeds.long()], (hash_seed << 32) + k).clone())
    return torch.stack(seen)[:, 0].tolist() if seen else []
