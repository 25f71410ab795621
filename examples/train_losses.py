#!/usr/bin/env python3
"""A small language model trained with the operators next to the shard step, on
one GPU: embedding lookup -> residual MLP blocks -> head -> policy or preference
loss -> gradients -> Muon for the blocks' matrices, AdamW for embedding and head.

  python examples/train_losses.py [--loss policy|preference] [--steps N]

The task is to answer token t with (7 t + 3) mod vocab.  With the policy loss the
model samples its answers and is rewarded for the right ones; with the preference
loss it is shown pairs of a right and a random answer.  Matrix products of the
model itself are torch's.  Prints the mean probability of the right answer.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixed_precision_zero_amd import binding as B  # noqa: E402
from mixed_precision_zero_amd import ops  # noqa: E402
from mixed_precision_zero_amd.muon import MuonStep, rms_lr_scale  # noqa: E402
from mixed_precision_zero_amd.shard import ShardStep  # noqa: E402


class Model:
    """Embedding, `blocks` of x + W2 relu(W1 x), head; bf16 weights, K
    micro-batches a step."""

    def __init__(self, vocab=64, dim=128, hidden=256, blocks=2, n_micro=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, scale: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
        self.vocab, self.dim, self.n_micro = vocab, dim, n_micro
        self.scale = math.sqrt(dim)
        shapes = [(hidden, dim), (dim, hidden)] * blocks
        self.blocks = MuonStep(shapes, n_micro, lr_scale=rms_lr_scale(shapes))
        self.blocks.load_master([rand(*s, scale=1 / math.sqrt(s[1])) for s in shapes])
        # embedding and head: AdamW on an externally filled accumulator
        self.ends = ShardStep([(vocab, dim), (vocab, dim)], 1, 0, 1)
        ends = [rand(vocab, dim, scale=1 / self.scale), rand(vocab, dim, scale=0.5 / self.scale)]
        self.ends.scatter_to_arena(self.ends.master, ends)
        self.ends.load_weights(ends)
        off, n = self.ends.arena_off, vocab * dim
        self.acc = [self.ends.acc[int(o):int(o) + n].view(vocab, dim) for o in off]
        self.d_pairs = torch.zeros(2, 2, dtype=torch.float64, device="cuda")
        self.d_S = torch.zeros(1, dtype=torch.float64, device="cuda")
        self.workspace = None

    def forward(self, ids):
        """Logits, and what the backward pass needs."""
        x = torch.empty(ids.numel(), self.dim, device="cuda", dtype=torch.bfloat16)
        ops.z1_embed_lookup(self.ends.weights[0], ids, x, scale=self.scale)
        saved = []
        for w1, w2 in zip(self.blocks.weights[0::2], self.blocks.weights[1::2]):
            a = torch.relu(x @ w1.t())
            saved.append((x, a))
            x = x + a @ w2.t()
        return x @ self.ends.weights[1].t(), (ids, saved, x)

    def backward(self, k, dlogits, saved):
        """Gradients of micro-batch k: the blocks' into bf16 slot k, those of
        embedding and head onto the fp32 accumulator."""
        ids, layers, x = saved
        head = dlogits.t().float() @ x.float()
        self.acc[1].copy_(head) if k == 0 else self.acc[1].add_(head)
        dx = dlogits @ self.ends.weights[1]
        for i in reversed(range(len(layers))):
            x, a = layers[i]
            w1, w2 = self.blocks.weights[2 * i], self.blocks.weights[2 * i + 1]
            self.blocks.grads[k][2 * i + 1].copy_(dx.t() @ a)
            da = (dx @ w2) * (a > 0)
            self.blocks.grads[k][2 * i].copy_(da.t() @ x)
            dx = dx + da @ w1
        need = ops.z1_embed_grad_workspace(ids.numel(), self.vocab, self.dim)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, device="cuda", dtype=torch.uint8)
        ops.z1_embed_grad(ids, dx, self.acc[0], scale=self.scale, accumulate=k > 0, workspace=self.workspace)

    def update(self, lr, clip=1.0, weight_decay=0.01):
        """One optimizer step on the accumulated gradients, clipped by the norm
        of the whole model."""
        self.blocks.accumulate_range(0, self.n_micro)
        B.z1_grad_norm_sq_acc(self.ends.plan, self.ends.d_S)
        B.z1_grad_norm_sq_pair(self.blocks.plan, self.d_pairs[0])
        B.z1_grad_norm_sq_pair(self.ends.plan, self.d_pairs[1])
        B.z1_norm_combine(self.d_pairs, 2, self.d_S)
        self.ends.d_S.copy_(self.d_S)
        self.blocks.update(d_S=self.d_S, lr=lr, momentum=0.95, weight_decay=weight_decay, clip=clip)
        self.ends.adamw(dict(lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=weight_decay, clip=clip))

    def close(self):
        self.blocks.close()
        self.ends.close()


def answer(ids, vocab):
    return (7 * ids + 3) % vocab


def policy_micro(model, k, ids, g):
    """Samples answers, rewards them and backpropagates the clipped policy loss
    with a KL term to the uniform policy."""
    n = ids.numel()
    logits, saved = model.forward(ids)
    picked = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=g)[:, 0]
    right = picked == answer(ids, model.vocab)
    adv = right.float() * model.vocab - 1.0
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    old, loss, token = f(n), f(1), f(n)
    ops.z1_token_logprob(logits, picked, old)
    ref = torch.full((n,), -math.log(model.vocab), device="cuda")
    ops.z1_policy_loss(logits, picked, old, adv / model.vocab, ref_logp=ref, kl_coef=1e-3,
                       scale=1.0 / (n * model.n_micro), loss=loss, token_loss=token, dlogits=logits)
    model.backward(k, logits, saved)
    return loss


def preference_micro(model, k, ids, g, length=4, beta=0.5):
    """Pairs of answers of `length` tokens each, a right one and a random one."""
    pairs = ids.numel() // length
    ids = ids[:pairs * length]
    rows = torch.stack([ids.view(pairs, length)] * 2, 1).reshape(-1)
    y = answer(ids, model.vocab).view(pairs, length)
    wrong = torch.randint(0, model.vocab, (pairs, length), generator=g, device="cuda")
    targets = torch.stack([y, wrong], 1).reshape(-1).contiguous()
    cu = torch.arange(2 * pairs + 1, device="cuda") * length
    logits, saved = model.forward(rows)
    n = rows.numel()
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    logp, lse, dlogp, loss, pair = f(n), f(n), f(n), f(1), f(pairs)
    ref = torch.full((n,), -math.log(model.vocab), device="cuda")
    ops.z1_token_logprob(logits, targets, logp, lse)
    ops.z1_preference_loss(logp, ref, targets, cu, beta=beta, scale=1.0 / (pairs * model.n_micro),
                           loss=loss, pair_loss=pair, dlogp=dlogp)
    ops.z1_logprob_grad(logits, targets, lse, dlogp, logits)
    model.backward(k, logits, saved)
    return loss


def right_probability(model):
    ids = torch.arange(model.vocab, device="cuda")
    logits, _ = model.forward(ids)
    logp = torch.empty(model.vocab, device="cuda")
    ops.z1_token_logprob(logits, answer(ids, model.vocab), logp)
    return float(logp.exp().mean())


def train(loss="policy", steps=100, tokens=1024, lr=2e-3, seed=0, report=None, **sizes):
    """Mean probability of the right answer before and after."""
    model = Model(seed=seed, **sizes)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    micro = {"policy": policy_micro, "preference": preference_micro}[loss]
    first = right_probability(model)
    for step in range(steps):
        for k in range(model.n_micro):
            ids = torch.randint(0, model.vocab, (tokens,), generator=g, device="cuda")
            value = micro(model, k, ids, g)
        model.update(lr)
        if report and (step + 1) % report == 0:
            print(f"step {step + 1}: loss {float(value):.4f}, right answers {right_probability(model):.3f}", flush=True)
    last = right_probability(model)
    model.close()
    return first, last


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("policy", "preference"), default="policy")
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    torch.cuda.set_device(0)
    print("right answers %.3f -> %.3f" % train(a.loss, a.steps, report=20))
