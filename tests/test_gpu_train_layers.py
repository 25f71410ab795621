"""The layers run together, as examples/train_layers.py trains with them: the
gradients of a whole model against its formula in 64 bits and against differences."""
import importlib.util
import math
import os

import pytest
import torch

import layer_refs as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(vocab=50, dim=72, heads=6, kv_heads=2, head_dim=16, hidden=88, blocks=2, n_micro=2)
# Steps between the loss and a weight's gradient: at most 14 a block and direction, and
# the head's, each off by at most its depth (88 here, 100 tokens for weights) times half
# a step of fp32 of its norm; the map of norms from step to step is that of residual
# sums, about one.
TOL = 60 * 100 * R.U32
# With bf16 between the steps each adds half a step of bf16.
TOL_BF16 = 60 * 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("train_layers", os.path.join(ROOT, "examples", "train_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rotate(x, angle):
    h = x.shape[-1] // 2
    a, b, c, s = x[..., :h], x[..., h:], angle.cos()[:, None], angle.sin()[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _normed(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def _loss(sizes, matrices, others, ids, targets, seed, offset, p):
    """The mean loss of one micro-batch in 64 bits on the CPU."""
    seqs, length = ids.shape
    h, g, d = sizes["heads"], sizes["kv_heads"], sizes["head_dim"]
    inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    angle = torch.arange(length, dtype=torch.float64).repeat(seqs)[:, None] * inv
    x = others[0][ids.flatten()] * math.sqrt(sizes["dim"])
    later = torch.ones(length, length, dtype=torch.bool).triu(1)
    for i in range(sizes["blocks"]):
        w_qkv, w_out, w_gate, w_up, w_down = matrices[5 * i:5 * i + 5]
        bias, q_norm, k_norm = others[2 + 3 * i:5 + 3 * i]
        q, k, v = (x @ w_qkv.t() + bias).split([h * d, g * d, g * d], 1)
        q = _rotate(_normed(q.unflatten(1, (h, d)), q_norm), angle)
        k = _rotate(_normed(k.unflatten(1, (g, d)), k_norm), angle)
        v = v.unflatten(1, (g, d))
        q, k, v = (t.unflatten(0, (seqs, length)).transpose(1, 2) for t in (q, k, v))
        k, v = (t.repeat_interleave(h // g, 1) for t in (k, v))
        att = torch.softmax((q @ k.transpose(2, 3) / math.sqrt(d)).masked_fill(later, -math.inf), 3) @ v
        o = att.transpose(1, 2).flatten(2).flatten(0, 1)
        x = x + R.drop(o @ w_out.t(), seed, offset + 2 * i, p)
        a = torch.nn.functional.silu(x @ w_gate.t()) * (x @ w_up.t())
        x = x + R.drop(a @ w_down.t(), seed, offset + 2 * i + 1, p)
    logp = torch.log_softmax(x @ others[1].t(), 1)
    return -logp.gather(1, targets.flatten()[:, None]).mean()


def _whole(model, matrices, others, batches, p):
    """The step's loss, as the micro-batches share it."""
    seed = int(model.rng[0])
    parts = [_loss(SIZES, matrices, others, ids.cpu(), targets.cpu(), seed, k * 2 * model.n_blocks, p)
             for k, (ids, targets) in enumerate(batches)]
    return sum(parts) / len(parts)


def _run(example, dtype, drop):
    """A model, its batches, the loss, and its gradients (matrices, others)."""
    model = example.Model(dtype=dtype, drop=drop, seed=3, **SIZES)
    g = torch.Generator(device="cuda").manual_seed(7)
    batches = [example.runs(SIZES["vocab"], 4, 25, g) for _ in range(SIZES["n_micro"])]
    loss = sum(float(model.micro(k, *b)) for k, b in enumerate(batches))
    grads = [sum(s[i].double() for s in model.grads).cpu() for i in range(len(model.matrices))]
    grads += [a.double().cpu() for a in model.acc]
    model.close()
    return model, batches, loss, grads


@pytest.mark.parametrize("drop", [0.0, 0.1])
def test_gradients_of_the_model(example, drop):
    model, batches, loss, got = _run(example, torch.float32, drop)
    leaves = [w.double().cpu().requires_grad_() for w in model.matrices + model.others]
    n = len(model.matrices)
    want = _whole(model, leaves[:n], leaves[n:], batches, drop)
    want.backward()
    assert abs(loss - want.item()) <= TOL * want.item()
    for i, (a, w) in enumerate(zip(got, leaves)):
        assert a.shape == w.shape
        assert float((a - w.grad).norm()) <= TOL * float(w.grad.norm()), i
    # differences of the loss along a direction that all weights move in
    g = torch.Generator().manual_seed(1)
    by = [torch.randn(w.shape, generator=g, dtype=torch.float64) * w.detach().abs().mean() for w in leaves]
    step = 1e-5
    with torch.no_grad():
        up, down = (float(_whole(model, *(lambda v: (v[:n], v[n:]))([w + s * b for w, b in zip(leaves, by)]), batches, drop))
                    for s in (step, -step))
    along = sum(float((a * b).sum()) for a, b in zip(got, by))
    # the gradients' own errors, and the third derivative's share of the difference
    most = sum(float(a.norm() * b.norm()) for a, b in zip(got, by))
    assert abs((up - down) / (2 * step) - along) <= (TOL + 1e-6) * most


def test_gradients_in_bf16(example):
    """The same with bf16 activations, weights' gradients in the step's slots."""
    _, _, want_loss, want = _run(example, torch.float32, 0.1)
    model, _, loss, got = _run(example, torch.bfloat16, 0.1)
    assert model.grads is model.blocks.grads
    assert abs(loss - want_loss) <= TOL_BF16 * want_loss
    for i, (a, b) in enumerate(zip(got, want)):
        assert float((a - b).norm()) <= TOL_BF16 * float(b.norm()), i


def test_the_example_runs(example):
    losses = example.train(steps=3, seqs=4, length=16)
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)


def test_a_step_takes_the_gradients(example):
    """Norm and update go on from what the layers left in slots and accumulator."""
    model = example.Model(drop=0.1, **SIZES)
    g = torch.Generator(device="cuda").manual_seed(5)
    for k in range(SIZES["n_micro"]):
        model.micro(k, *example.runs(SIZES["vocab"], 4, 25, g))
    S = sum(float(sum(s[i].float() for s in model.grads).double().square().sum()) for i in range(len(model.matrices)))
    S += sum(float(a.double().square().sum()) for a in model.acc)
    before = [w.clone() for w in model.matrices + model.others]
    model.update(2e-3)
    torch.cuda.synchronize()
    assert abs(float(model.d_S) - S) <= 1e-12 * S
    # 2e-3 is several steps of bf16 for most of these weights
    assert all(not torch.equal(a, b) for a, b in zip(before, model.matrices + model.others))
    assert all(torch.isfinite(w).all() for w in model.matrices + model.others)
    model.close()
