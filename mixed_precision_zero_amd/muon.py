"""One rank's Muon step: the buffers of its matrices wired to a libz1 plan and
a Muon handle.

The hidden matrices of a model are updated by Muon, everything else (embedding,
head, norm weights) by the AdamW of ``shard.ShardStep``.  The orthogonalisation
needs whole matrices, so the ranks share out matrices instead of slices
(``assign_matrices``), and the plan of a rank's own matrices is one with
dp_size 1.  The gradient path is the shard step's: bf16 micro-batch gradients
accumulated in fp32, the exactly rounded norm, clipping read on the device.

As in ``shard``, this is memory plumbing; no arithmetic of the step happens
here.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence

import torch

from . import binding as B
from . import ops
from .shard import flat_views


def assign_matrices(shapes: Sequence[Sequence[int]], dp_size: int) -> List[int]:
    """The rank that owns each matrix: largest first to the least loaded rank
    (the lowest of equals), the load being the products' multiply-adds
    3 m^2 n + m^3 (m <= n) of one Newton-Schulz step."""
    if dp_size < 1:
        raise ValueError(f"dp_size {dp_size}")
    cost = []
    for s in shapes:
        if len(s) != 2:
            raise ValueError(f"shape {tuple(s)}: expected a matrix")
        m, n = sorted(int(x) for x in s)
        cost.append(3 * m * m * n + m ** 3)
    load = [0] * dp_size
    owner = [0] * len(cost)
    for i in sorted(range(len(cost)), key=lambda i: (-cost[i], i)):
        r = min(range(dp_size), key=lambda r: (load[r], r))
        owner[i] = r
        load[r] += cost[i]
    return owner


def rms_lr_scale(shapes: Sequence[Sequence[int]], rms: float = 0.2) -> List[float]:
    """Per-matrix lr_scale that gives an orthogonalised update (singular values
    near 1, root mean square 1 / sqrt(max side)) the root mean square `rms`, so
    that one learning rate serves Muon and AdamW."""
    return [rms * math.sqrt(max(int(s[0]), int(s[1]))) for s in shapes]


class MuonStep:
    """Buffers and handles of the matrices one rank owns.  master, momentum and
    acc are fp32 arenas in the plan's order, weights and grads[k] bf16 tensors
    of the given shapes.  wide: as in ops.z1_muon_create."""

    def __init__(self, shapes: Sequence[Sequence[int]], n_micro: int, device="cuda",
                 weights: Optional[List[torch.Tensor]] = None,
                 grads: Optional[List[List[torch.Tensor]]] = None,
                 lr_scale: Optional[Sequence[float]] = None,
                 wd_scale: Optional[Sequence[float]] = None, ns_steps: int = 5,
                 coeffs=ops.MUON_COEFFS, eps: float = 1e-7, wide: bool = False):
        self.shapes = [tuple(int(x) for x in s) for s in shapes]
        self.numel = [m * n for m, n in self.shapes]
        self.n_micro = n_micro
        self.device = torch.device(device)
        _, _, self.arena_off, total = B.z1_shard_plan(self.numel, 1, 0)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.master = torch.zeros(total, **f32)
        self.momentum = torch.zeros(total, **f32)
        self.acc = torch.zeros(total, **f32)
        bf = dict(dtype=torch.bfloat16, device=self.device)
        self.weights = weights if weights is not None else flat_views(self.shapes, **bf)
        self.grads = grads if grads is not None else [flat_views(self.shapes, **bf)
                                                      for _ in range(n_micro)]
        self.d_S = torch.zeros(1, dtype=torch.float64, device=self.device)
        # only the plan's accumulation and norm run, which touch acc alone: the
        # momentum stands in for AdamW's two moments
        self.plan = B.z1_plan_create(self.numel, 1, 0, self.weights, self.grads, self.master,
                                     self.momentum, self.momentum, self.acc)
        self.muon = ops.z1_muon_create(self.shapes, self.views(self.acc),
                                       momentum=self.views(self.momentum),
                                       master=self.views(self.master), weights=self.weights,
                                       lr_scale=lr_scale, wd_scale=wd_scale, ns_steps=ns_steps,
                                       coeffs=coeffs, eps=eps, wide=wide)

    def views(self, arena: torch.Tensor) -> List[torch.Tensor]:
        """The matrices of an arena."""
        return [arena[int(o):int(o) + n].view(s)
                for o, n, s in zip(self.arena_off, self.numel, self.shapes)]

    def load_master(self, full: Sequence[torch.Tensor]) -> None:
        """The fp32 master and the bf16 weights from full tensors."""
        for v, w, x in zip(self.views(self.master), self.weights, full):
            v.copy_(x)
            w.copy_(x)

    def accumulate(self, k: int, stream=None) -> None:
        B.z1_accum_grads(self.plan, k, stream)

    def accumulate_range(self, k_begin: int, k_end: int, stream=None) -> None:
        B.z1_accum_grads_range(self.plan, k_begin, k_end, stream)

    def norm(self, stream=None) -> None:
        """d_S: the squared gradient norm of these matrices alone."""
        B.z1_grad_norm_sq(self.plan, self.d_S, stream)

    def update(self, *, d_S=None, stream=None, **hp) -> None:
        """z1_muon_step; d_S: the squared norm clipping goes by (default: of
        these matrices alone; pass that of the whole model)."""
        ops.z1_muon_step(self.muon, d_S=self.d_S if d_S is None else d_S, stream=stream, **hp)

    def step(self, stream=None, **hp) -> None:
        """Accumulation of every micro-batch slot, norm and update."""
        self.accumulate_range(0, self.n_micro, stream)
        self.norm(stream)
        self.update(stream=stream, **hp)

    def close(self) -> None:
        self.muon.close()
        self.plan.close()
