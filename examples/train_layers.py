#!/usr/bin/env python3
"""A small transformer trained on one GPU with its layers on the kernels next to the
shard step: embedding -> blocks of (projections, query-key norm and rotation,
attention, output projection, gated MLP, dropout) -> head -> next-token loss ->
gradients -> Muon for the blocks' matrices, AdamW for the rest.

  python examples/train_layers.py [--steps N]

The matrices' gradients go into the bf16 micro-batch slots of the step, those of
embedding, head, biases and norm weights straight onto its fp32 accumulator.
Attention itself is torch's.  The data are runs of (7 t + 3) mod vocab; prints the
mean loss as it goes.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixed_precision_zero_amd import binding as B  # noqa: E402
from mixed_precision_zero_amd import layers, ops  # noqa: E402
from mixed_precision_zero_amd.muon import MuonStep, rms_lr_scale  # noqa: E402
from mixed_precision_zero_amd.shard import ShardStep  # noqa: E402


class Model:
    """`blocks` of attention and gated MLP; bf16 weights, n_micro micro-batches a
    step.  With dtype fp32 activations and gradients are fp32, and weights the bf16
    ones' values; that is for checks of the gradients and takes no update."""

    def __init__(self, vocab=64, dim=128, heads=4, kv_heads=2, head_dim=32, hidden=192, blocks=2, n_micro=2,
                 drop=0.1, seed=0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, scale: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
        self.vocab, self.dim, self.heads, self.kv_heads, self.head_dim = vocab, dim, heads, kv_heads, head_dim
        self.n_micro, self.n_blocks, self.drop, self.dtype = n_micro, blocks, drop, dtype
        self.scale = math.sqrt(dim)
        self.qkv = (heads + 2 * kv_heads) * head_dim
        shapes = [(self.qkv, dim), (dim, heads * head_dim), (hidden, dim), (hidden, dim), (dim, hidden)] * blocks
        self.blocks = MuonStep(shapes, n_micro, lr_scale=rms_lr_scale(shapes))
        self.blocks.load_master([rand(*s, scale=1 / math.sqrt(s[1])) for s in shapes])
        # embedding, head, and each block's bias and norm weights: AdamW on an
        # externally filled accumulator
        small = [(vocab, dim), (vocab, dim)] + [(self.qkv,), (head_dim,), (head_dim,)] * blocks
        self.rest = ShardStep(small, 1, 0, 1)
        full = [rand(vocab, dim, scale=1 / self.scale), rand(vocab, dim, scale=0.5 / self.scale)]
        for _ in range(blocks):
            full += [rand(self.qkv, scale=0.1), 1 + rand(head_dim, scale=0.1), 1 + rand(head_dim, scale=0.1)]
        self.rest.scatter_to_arena(self.rest.master, full)
        self.rest.load_weights(full)
        self.acc = [self.rest.acc[int(o):int(o) + math.prod(s)].view(s) for o, s in zip(self.rest.arena_off, small)]
        self.d_pairs = torch.zeros(2, 2, dtype=torch.float64, device="cuda")
        self.d_S = torch.zeros(1, dtype=torch.float64, device="cuda")
        self.inv_freq = 10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64, device="cuda") / head_dim)
        # (seed, offset) of the dropouts; the offset moves on with every micro-batch
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
        self.work = torch.empty(0, device="cuda", dtype=torch.uint8)
        if dtype == torch.float32:
            self.grads = [[torch.zeros(s, device="cuda") for s in shapes] for _ in range(n_micro)]
            self.matrices = [w.float() for w in self.blocks.weights]
            self.others = [w.float() for w in self.rest.weights]
        else:
            self.grads, self.matrices, self.others = self.blocks.grads, self.blocks.weights, self.rest.weights

    def _new(self, *shape):
        return torch.empty(*shape, device="cuda", dtype=self.dtype)

    def _room(self, need):
        """A workspace of `need` bytes; one serves every call of the stream in turn."""
        if self.work.numel() < need:
            self.work = torch.empty(need, device="cuda", dtype=torch.uint8)
        return self.work

    def _linear(self, x, w, **more):
        y = self._new(x.shape[0], w.shape[0])
        layers.z1_linear(x, w, y, workspace=self._room(layers.z1_linear_workspace(x, w)), **more)
        return y

    def _linear_grad(self, dz, x, w, dweight, accumulate=False, add=None):
        dx = self._new(*x.shape)
        layers.z1_linear_grad(dz, x, w, dx=dx, add=add, dweight=dweight, accumulate=accumulate,
                              workspace=self._room(layers.z1_linear_grad_workspace(dz, x, w)))
        return dx

    def _dropout(self, block, site):
        return layers.Dropout(self.rng, self.drop, 2 * block + site) if self.drop else None

    def _undrop(self, dy, drop):
        """The gradient in front of a dropout."""
        if drop is None:
            return dy
        dz = self._new(*dy.shape)
        layers.z1_linear_dz(dy, dz, dropout=drop)
        return dz

    def _heads(self, qkv):
        """q, k and v [tokens, heads, head_dim] as views of the projections."""
        h, g, d = self.heads, self.kv_heads, self.head_dim
        q, k, v = qkv.split([h * d, g * d, g * d], 1)
        return q.unflatten(1, (h, d)), k.unflatten(1, (g, d)), v.unflatten(1, (g, d))

    def _per_head(self, t, seqs):
        """[tokens, heads, dim] in fp32 as [sequences * heads, length, dim], keys and
        values of shared heads repeated."""
        t = t.float().unflatten(0, (seqs, -1)).transpose(1, 2)
        return t.repeat_interleave(self.heads // t.shape[1], 1).flatten(0, 1).contiguous()

    def _per_token(self, t, seqs, heads):
        """The way back; the gradients of a shared head are added up."""
        t = t.unflatten(0, (seqs, heads, -1)).sum(2).transpose(1, 2)
        return t.flatten(0, 1)

    def _attention(self, q, k, v, seqs):
        q, k, v = (self._per_head(t, seqs) for t in (q, k, v))
        s = torch.bmm(q, k.transpose(1, 2)) / math.sqrt(self.head_dim)
        later = torch.ones(s.shape[1:], dtype=torch.bool, device="cuda").triu(1)
        p = torch.softmax(s.masked_fill(later, -math.inf), 2)
        o = self._per_token(torch.bmm(p, v), seqs, self.heads).flatten(1).to(self.dtype)
        return o, (q, k, v, p)

    def _attention_grad(self, do, saved, seqs):
        q, k, v, p = saved
        do = self._per_head(do.unflatten(1, (self.heads, self.head_dim)), seqs)
        dp = torch.bmm(do, v.transpose(1, 2))
        ds = p * (dp - (dp * p).sum(2, keepdim=True)) / math.sqrt(self.head_dim)
        back = lambda t, heads: self._per_token(t, seqs, heads).to(self.dtype).contiguous()  # noqa: E731
        return (back(torch.bmm(ds, k), self.heads), back(torch.bmm(ds.transpose(1, 2), q), self.kv_heads),
                back(torch.bmm(p.transpose(1, 2), do), self.kv_heads))

    def forward(self, ids):
        """Logits of ids [sequences, length], and what the backward pass needs."""
        seqs, length = ids.shape
        pos = torch.arange(length, device="cuda").repeat(seqs)
        x = self._new(ids.numel(), self.dim)
        ops.z1_embed_lookup(self.others[0], ids.flatten(), x, scale=self.scale)
        saved = []
        for i in range(self.n_blocks):
            w_qkv, w_out, w_gate, w_up, w_down = self.matrices[5 * i:5 * i + 5]
            bias, q_norm, k_norm = self.others[2 + 3 * i:5 + 3 * i]
            qkv = self._linear(x, w_qkv, bias=bias)
            q, k, v = self._heads(qkv)
            qr, kr = self._new(*q.shape), self._new(*k.shape)
            layers.z1_qk_norm_rope(q, k, qr, kr, pos, self.inv_freq, q_weight=q_norm, k_weight=k_norm)
            o, att = self._attention(qr, kr, v, seqs)
            x1 = self._linear(o, w_out, residual=x, dropout=self._dropout(i, 0))
            up = self._linear(x1, w_up)
            pre = self._new(*up.shape)
            a = self._linear(x1, w_gate, act="silu", mul=up, pre=pre)
            x2 = self._linear(a, w_down, residual=x1, dropout=self._dropout(i, 1))
            saved.append((x, qkv, att, o, x1, up, pre, a))
            x = x2
        return self._linear(x, self.others[1]), (ids, pos, saved, x)

    def backward(self, k, dlogits, saved):
        """Gradients of micro-batch k."""
        ids, pos, saved, x = saved
        seqs = ids.shape[0]
        grads, more = self.grads[k], dict(accumulate=k > 0)
        dx = self._linear_grad(dlogits, x, self.others[1], self.acc[1], **more)
        for i in reversed(range(self.n_blocks)):
            x, qkv, att, o, x1, up, pre, a = saved[i]
            w_qkv, w_out, w_gate, w_up, w_down = self.matrices[5 * i:5 * i + 5]
            g_qkv, g_out, g_gate, g_up, g_down = grads[5 * i:5 * i + 5]
            _, q_norm, k_norm = self.others[2 + 3 * i:5 + 3 * i]
            a_bias, a_q, a_k = self.acc[2 + 3 * i:5 + 3 * i]
            da = self._linear_grad(self._undrop(dx, self._dropout(i, 1)), a, w_down, g_down)
            dgate, dup = self._new(*pre.shape), self._new(*up.shape)
            layers.z1_linear_dz(da, dgate, act="silu", pre=pre, mul=up, dmul=dup)
            dx = self._linear_grad(dgate, x1, w_gate, g_gate, add=dx)
            dx = self._linear_grad(dup, x1, w_up, g_up, add=dx)
            do = self._linear_grad(self._undrop(dx, self._dropout(i, 0)), o, w_out, g_out)
            dq, dk, dv = self._attention_grad(do, att, seqs)
            dqkv = self._new(*qkv.shape)
            (q, kk, _), (tq, tk, tv) = self._heads(qkv), self._heads(dqkv)
            tv.copy_(dv)
            need = layers.z1_qk_norm_rope_grad_workspace(len(pos), self.heads, self.kv_heads, self.head_dim)
            layers.z1_qk_norm_rope_grad(q, kk, dq, dk, tq, tk, pos, self.inv_freq, q_weight=q_norm, k_weight=k_norm,
                                        dq_weight=a_q, dk_weight=a_k, workspace=self._room(need), **more)
            need = layers.z1_linear_dz_workspace(len(pos), self.qkv)
            layers.z1_linear_dz(dqkv, dbias=a_bias, workspace=self._room(need), **more)
            dx = self._linear_grad(dqkv, x, w_qkv, g_qkv, add=dx)
        need = ops.z1_embed_grad_workspace(ids.numel(), self.vocab, self.dim)
        ops.z1_embed_grad(ids.flatten(), dx, self.acc[0], scale=self.scale, workspace=self._room(need), **more)

    def micro(self, k, ids, targets):
        """One micro-batch: its share of the mean loss over the step's tokens, and
        its gradients."""
        n = ids.numel()
        logits, saved = self.forward(ids)
        logp, lse = (torch.empty(n, device="cuda") for _ in range(2))
        ops.z1_token_logprob(logits, targets.flatten(), logp, lse)
        dlogp = torch.full((n,), -1.0 / (n * self.n_micro), device="cuda")
        ops.z1_logprob_grad(logits, targets.flatten(), lse, dlogp, logits)
        self.backward(k, logits, saved)
        self.rng[1] += 2 * self.n_blocks
        return -logp.mean() / self.n_micro

    def update(self, lr, clip=1.0, weight_decay=0.01):
        """One optimizer step on the accumulated gradients, clipped by the norm of
        the whole model."""
        self.blocks.accumulate_range(0, self.n_micro)
        B.z1_grad_norm_sq_acc(self.rest.plan, self.rest.d_S)
        B.z1_grad_norm_sq_pair(self.blocks.plan, self.d_pairs[0])
        B.z1_grad_norm_sq_pair(self.rest.plan, self.d_pairs[1])
        B.z1_norm_combine(self.d_pairs, 2, self.d_S)
        self.rest.d_S.copy_(self.d_S)
        self.blocks.update(d_S=self.d_S, lr=lr, momentum=0.95, weight_decay=weight_decay, clip=clip)
        self.rest.adamw(dict(lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=weight_decay, clip=clip))

    def close(self):
        self.blocks.close()
        self.rest.close()


def runs(vocab, seqs, length, g):
    """Inputs and targets: t, 7 t + 3, ... from random starts."""
    t = [torch.randint(0, vocab, (seqs,), generator=g, device="cuda")]
    for _ in range(length):
        t.append((7 * t[-1] + 3) % vocab)
    t = torch.stack(t, 1)
    return t[:, :-1].contiguous(), t[:, 1:].contiguous()


def train(steps=100, seqs=16, length=32, lr=2e-3, seed=0, report=None, **sizes):
    """The mean loss of every step."""
    model = Model(seed=seed, **sizes)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = []
    for step in range(steps):
        parts = [model.micro(k, *runs(model.vocab, seqs, length, g)) for k in range(model.n_micro)]
        model.update(lr)
        losses.append(float(sum(parts)))
        if report and (step + 1) % report == 0:
            print(f"step {step + 1}: loss {losses[-1]:.4f}", flush=True)
    model.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    torch.cuda.set_device(0)
    train(a.steps, report=20)
