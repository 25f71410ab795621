"""The operators run together: MuonStep over the shard step's accumulation, and
examples/train_losses.py."""
import importlib.util
import os

import pytest
import torch

from mixed_precision_zero_amd import binding as B
from mixed_precision_zero_amd import ops as O
from mixed_precision_zero_amd.muon import MuonStep, rms_lr_scale

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _example():
    spec = importlib.util.spec_from_file_location("train_losses", os.path.join(ROOT, "examples", "train_losses.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_muon_step_over_the_accumulated_gradient():
    """Two steps of K micro-batches: acc and S are the shard step's, the update
    is that of a handle bound to the same values directly, bit for bit."""
    shapes, K = [(64, 96), (300, 130), (7, 33)], 3
    hp = dict(lr=1e-2, momentum=0.9, weight_decay=0.1, nesterov=True, clip=0.05)
    g = torch.Generator(device="cuda").manual_seed(0)
    st = MuonStep(shapes, K, lr_scale=rms_lr_scale(shapes))
    full = [torch.randn(s, generator=g, device="cuda") * 0.02 for s in shapes]
    st.load_master(full)
    acc = [torch.zeros(s, device="cuda") for s in shapes]
    mom, master = [torch.zeros(s, device="cuda") for s in shapes], [x.clone() for x in full]
    w = [x.bfloat16() for x in full]
    direct = O.z1_muon_create(shapes, acc, momentum=mom, master=master, weights=w, lr_scale=rms_lr_scale(shapes))
    for step in range(2):
        for k in range(K):
            for t in st.grads[k]:
                t.copy_(torch.randn(t.shape, generator=g, device="cuda") * 1e-3)
        for i in range(len(shapes)):
            acc[i].copy_(st.grads[0][i].float())
            for k in range(1, K):
                acc[i].add_(st.grads[k][i].float())
        S = torch.stack([a.double().square().sum() for a in acc]).sum().reshape(1)
        st.step(**hp)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(st.views(st.acc), acc))
        assert abs(float(st.d_S) - float(S)) <= 1e-12 * float(S)
        O.z1_muon_step(direct, d_S=st.d_S, **hp)
        torch.cuda.synchronize()
        for a, b in ((st.views(st.momentum), mom), (st.views(st.master), master), (st.weights, w)):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), step
        assert not torch.equal(master[0], full[0])
    st.close()
    direct.close()


def test_norm_of_the_whole_model_reaches_muon():
    """S from the norm exchange of two plans clips both parts alike."""
    shapes = [(64, 64)]
    st = MuonStep(shapes, 1)
    st.grads[0][0].fill_(2.0 ** -6)
    d_S = torch.tensor([4.0], dtype=torch.float64, device="cuda")
    st.accumulate(0)
    st.norm()
    st.update(d_S=d_S, lr=1.0, momentum=0.5, nesterov=False, clip=1.0)
    torch.cuda.synchronize()
    c = torch.tensor(1.0 / (2.0 + 1e-6), dtype=torch.float64).float()
    assert torch.equal(st.views(st.momentum)[0], torch.full((64, 64), 2.0 ** -6, device="cuda") * c.cuda())
    st.close()


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_example_learns_the_task(loss):
    m = _example()
    torch.cuda.set_device(0)
    first, last = m.train(loss, steps=40, tokens=512)
    assert first < 0.05 and last > 0.5, (first, last)


def test_embedding_gradient_feeds_the_shard_step():
    """Micro-batches summed straight onto the acc arena: the norm of an
    externally filled accumulator and AdamW go on from there."""
    m = _example()
    model = m.Model(vocab=50, dim=24, hidden=32, blocks=1, n_micro=2)
    g = torch.Generator(device="cuda").manual_seed(2)
    want = torch.zeros(50, 24, dtype=torch.float64, device="cuda")
    for k in range(2):
        ids = torch.randint(0, 50, (200,), generator=g, device="cuda")
        dx = torch.randn(200, 24, generator=g, device="cuda").bfloat16()
        ws = torch.empty(O.z1_embed_grad_workspace(200, 50, 24), device="cuda", dtype=torch.uint8)
        O.z1_embed_grad(ids, dx, model.acc[0], scale=model.scale, accumulate=k > 0, workspace=ws)
        want.index_add_(0, ids, dx.double() * model.scale)
    model.acc[1].zero_()
    B.z1_grad_norm_sq_acc(model.ends.plan, model.ends.d_S)
    torch.cuda.synchronize()
    off = model.acc[0].double() - want
    assert float(off.abs().max()) <= 220 * 2.0 ** -24 * float(want.abs().max())
    S = float(model.acc[0].double().square().sum())
    assert abs(float(model.ends.d_S) - S) <= 1e-12 * S
    model.close()
