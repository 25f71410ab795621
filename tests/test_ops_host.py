"""Host-side checks of the operators (include/z1_ops.h): symbols, refusals of
the C ABI and of the binding.  No GPU needed: every case is decided before any
device work."""
import ctypes
import os
import re

import pytest
import torch

from mixed_precision_zero_amd import binding as B
from mixed_precision_zero_amd import ops as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PP = ctypes.POINTER(ctypes.c_void_p)
PI = ctypes.POINTER(ctypes.c_int64)


def test_every_declared_symbol_is_exported():
    text = open(os.path.join(ROOT, "include", "z1_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(z1_[a-z_0-9]+)\s*\(", text))
    assert names == set(O.EXPORTS)
    for name in names:
        assert hasattr(B.lib, name)
    assert O.z1_ops_abi_version() == 1


def test_header_is_plain_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "z1_ops.h"\nint main(void) { z1_policy_args a; z1_muon_bind b; (void)a; (void)b; '
                   'return Z1_OPS_ABI_VERSION - 1; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "t.o")], check=True)


def test_structures_match_the_header(tmp_path):
    """Sizes of the ctypes structures against the C compiler's."""
    import subprocess
    names = {"z1_muon_bind": O.MuonBind, "z1_muon_hp": O.MuonHP, "z1_embed_args": O.EmbedArgs, "z1_logits": O.Logits,
             "z1_policy_args": O.PolicyArgs, "z1_preference_args": O.PreferenceArgs}
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include "z1_ops.h"\nint main(void) { printf("' + "%d " * len(names) + '", '
                   + ", ".join(f"(int)sizeof({n})" for n in names) + "); return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(s) for s in names.values()]


def muon_bind(**over):
    rows, cols = (ctypes.c_int64 * 2)(64, 3), (ctypes.c_int64 * 2)(32, 5)
    ptr = lambda base: (ctypes.c_void_p * 2)(base, base + 0x1000)  # noqa: E731
    arr = dict(grad=ptr(0x10000), momentum=ptr(0x20000), master=ptr(0x30000),
               weights=ptr(0x40000), ortho=ptr(0x50000))
    b = O.MuonBind(n=2, grad_dtype=0, rows=ctypes.cast(rows, PI), cols=ctypes.cast(cols, PI),
                   a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, ns_steps=5, reserved=0)
    for k, v in over.items():
        if k == "rows1":
            rows[1] = v
        elif k.startswith("at_"):
            arr[k[3:]][1] = v
        elif k in arr:
            arr[k] = v
        else:
            setattr(b, k, v)
    for k, v in arr.items():
        setattr(b, k, ctypes.cast(v, PP) if v is not None else None)
    return b, (rows, cols, arr)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), B.Z1_EINVAL), (dict(grad_dtype=2), B.Z1_EINVAL), (dict(grad_dtype=-1), B.Z1_EINVAL),
    (dict(rows1=0), B.Z1_EINVAL), (dict(rows1=(1 << 20) + 1), B.Z1_EINVAL), (dict(rows=None), B.Z1_EINVAL),
    (dict(ns_steps=0), B.Z1_EINVAL), (dict(ns_steps=33), B.Z1_EINVAL), (dict(eps=-1.0), B.Z1_EINVAL),
    (dict(eps=float("nan")), B.Z1_EINVAL), (dict(reserved=1), B.Z1_EINVAL), (dict(grad=None), B.Z1_EINVAL),
    (dict(master=None), B.Z1_EINVAL), (dict(momentum=None), B.Z1_EINVAL), (dict(weights=None), B.Z1_EINVAL),
    (dict(momentum=None, master=None, weights=None, ortho=None), B.Z1_EINVAL),
    (dict(at_grad=0), B.Z1_EINVAL), (dict(at_master=0), B.Z1_EINVAL), (dict(at_ortho=0), B.Z1_EINVAL),
    (dict(at_grad=0x10002), B.Z1_EALIGN), (dict(at_weights=0x40001), B.Z1_EALIGN),
    (dict(at_momentum=0x20001), B.Z1_EALIGN), (dict(at_ortho=0x50001), B.Z1_EALIGN),
    (dict(at_ortho=0x50001, at_master=0), B.Z1_EINVAL),         # a null pointer before an alignment
    (dict(a=float("inf")), B.Z1_EINVAL), (dict(a=4.0, b=0.0, c=0.0), B.Z1_EINVAL),   # |X| leaves the range
    (dict(a=1.0, b=-4.5, c=0.0, ns_steps=1), B.Z1_EINVAL),      # |b s + c s^2| = 4.5
    (dict(a=1.0, b=0.0, c=4.0, ns_steps=1), B.Z1_EINVAL),
])
def test_muon_create_refuses(over, status):
    b, keep = muon_bind(**over)
    h = ctypes.c_void_p(1)
    assert B.lib.z1_muon_create(ctypes.byref(h), ctypes.byref(b), None) == status
    assert h.value is None


def test_muon_coefficients_in_range_are_not_refused_for_their_range():
    """Without a GPU a valid bind gets as far as the device check (EINVAL);
    the range check itself is looked at through its only visible effect, the
    alignment error that comes after it."""
    for a, b, c, steps in ((3.4445, -4.7750, 2.0315, 5), (1.5, -0.5, 0.0, 10), (3.0, -3.2, 1.2, 8),
                           (1.0, 0.0, 0.0, 32)):
        bind, keep = muon_bind(a=a, b=b, c=c, ns_steps=steps, at_grad=0x10002)
        h = ctypes.c_void_p()
        assert B.lib.z1_muon_create(ctypes.byref(h), ctypes.byref(bind), None) == B.Z1_EALIGN


def test_null_handles():
    hp = O.MuonHP(1e-3, 0.95, 0.1, 0.0, 1, 0)
    assert B.lib.z1_muon_step(None, ctypes.byref(hp), None, None) == B.Z1_EINVAL
    assert B.lib.z1_muon_orthogonalize(None, None) == B.Z1_EINVAL
    assert B.lib.z1_muon_destroy(None) == B.Z1_OK
    assert B.lib.z1_muon_create(None, None, None) == B.Z1_EINVAL
    assert B.lib.z1_policy_loss(None, None, None) == B.Z1_EINVAL
    assert B.lib.z1_preference_loss(None, None) == B.Z1_EINVAL
    assert B.lib.z1_token_logprob(None, None, None, None) == B.Z1_EINVAL
    assert B.lib.z1_logprob_grad(None, None, None, None, 0, None) == B.Z1_EINVAL
    assert B.lib.z1_embed_lookup(None, None, 0, None, 0, None) == B.Z1_EINVAL
    assert B.lib.z1_embed_grad(None, None, 0, None, 0, None, 0, None) == B.Z1_EINVAL


def embed_args(**over):
    a = O.EmbedArgs(100, 50, 16, 0x1000, 0, 1, 1.0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(n_ids=-1), B.Z1_EINVAL), (dict(n_ids=(1 << 30) + 1), B.Z1_EINVAL), (dict(vocab=0), B.Z1_EINVAL),
    (dict(vocab=(1 << 24) + 1), B.Z1_EINVAL), (dict(dim=0), B.Z1_EINVAL), (dict(dim=(1 << 20) + 1), B.Z1_EINVAL),
    (dict(ids=None), B.Z1_EINVAL), (dict(id_type=2), B.Z1_EINVAL), (dict(dtype=3), B.Z1_EINVAL),
    (dict(scale=float("inf")), B.Z1_EINVAL), (dict(ids=0x1004), B.Z1_EALIGN),
])
def test_embed_refuses(over, status):
    a = embed_args(**over)
    assert B.lib.z1_embed_lookup(ctypes.byref(a), 0x2000, 16, 0x3000, 16, None) == status
    assert B.lib.z1_embed_grad(ctypes.byref(a), 0x2000, 16, 0x3000, 0, 0x4000, 1 << 40, None) == status


def test_embed_refuses_buffers():
    a = embed_args()
    need = O.z1_embed_grad_workspace(100, 50, 16)
    L = B.lib
    assert L.z1_embed_lookup(ctypes.byref(a), None, 16, 0x3000, 16, None) == B.Z1_EINVAL
    assert L.z1_embed_lookup(ctypes.byref(a), 0x2000, 15, 0x3000, 16, None) == B.Z1_EINVAL
    assert L.z1_embed_lookup(ctypes.byref(a), 0x2000, 16, 0x3000, 15, None) == B.Z1_EINVAL
    assert L.z1_embed_lookup(ctypes.byref(a), 0x2001, 16, 0x3000, 16, None) == B.Z1_EALIGN
    grad = lambda dout=0x2000, ld=16, dw=0x3000, acc=0, ws=0x4000, n=need: L.z1_embed_grad(  # noqa: E731
        ctypes.byref(a), dout, ld, dw, acc, ws, n, None)
    assert grad(dout=None) == grad(dw=None) == grad(ws=None) == B.Z1_EINVAL
    assert grad(ld=15) == grad(acc=2) == grad(n=need - 1) == B.Z1_EINVAL
    assert grad(dout=0x2001) == grad(dw=0x3002) == grad(ws=0x4008) == B.Z1_EALIGN
    assert L.z1_embed_grad_workspace(1, 1, 1, None) == B.Z1_EINVAL
    with pytest.raises(B.Z1Error):
        O.z1_embed_grad_workspace(1, 0, 1)


def logits_args(**over):
    x = O.Logits(4, 100, 0x10000, 100, 0x20000, 0, 1)
    for k, v in over.items():
        setattr(x, k, v)
    return x


@pytest.mark.parametrize("over,status", [
    (dict(n_rows=-1), B.Z1_EINVAL), (dict(n_rows=1 << 31), B.Z1_EINVAL), (dict(vocab=0), B.Z1_EINVAL),
    (dict(vocab=(1 << 30) + 1, ld=1 << 31), B.Z1_EINVAL), (dict(ld=99), B.Z1_EINVAL), (dict(dtype=3), B.Z1_EINVAL),
    (dict(target_type=-1), B.Z1_EINVAL), (dict(logits=None), B.Z1_EINVAL), (dict(targets=None), B.Z1_EINVAL),
    (dict(logits=0x10001), B.Z1_EALIGN), (dict(targets=0x20004), B.Z1_EALIGN),
])
def test_losses_refuse_logits(over, status):
    x = logits_args(**over)
    f = 0x30000
    p = O.PolicyArgs(f, f, f, f, 0.2, 0.2, 0.1, 1.0, f, f, f, f, 1 << 31)
    assert B.lib.z1_token_logprob(ctypes.byref(x), f, f, None) == status
    assert B.lib.z1_logprob_grad(ctypes.byref(x), f, f, f, 1 << 31, None) == status
    assert B.lib.z1_policy_loss(ctypes.byref(x), ctypes.byref(p), None) == status


def test_in_place_gradient_needs_the_same_rows():
    x = logits_args(ld=104)
    f = 0x30000
    p = O.PolicyArgs(f, f, f, f, 0.2, 0.2, 0.1, 1.0, f, f, f, 0x10000, 100)
    assert B.lib.z1_policy_loss(ctypes.byref(x), ctypes.byref(p), None) == B.Z1_EINVAL
    assert B.lib.z1_logprob_grad(ctypes.byref(x), f, f, 0x10000, 100, None) == B.Z1_EINVAL


@pytest.mark.parametrize("over,status", [
    (dict(clip_low=-0.1), B.Z1_EINVAL), (dict(clip_low=1.5), B.Z1_EINVAL), (dict(clip_high=-0.1), B.Z1_EINVAL),
    (dict(clip_high=float("inf")), B.Z1_EINVAL), (dict(kl_coef=float("nan")), B.Z1_EINVAL),
    (dict(scale=float("nan")), B.Z1_EINVAL), (dict(old_logp=None), B.Z1_EINVAL), (dict(advantages=None), B.Z1_EINVAL),
    (dict(loss=None), B.Z1_EINVAL), (dict(token_loss=None), B.Z1_EINVAL), (dict(ld_dlogits=99), B.Z1_EINVAL),
    (dict(old_logp=0x30002), B.Z1_EALIGN), (dict(weights=0x30002), B.Z1_EALIGN), (dict(dlogits=0x30001), B.Z1_EALIGN),
    (dict(loss=0x30002), B.Z1_EALIGN),
])
def test_policy_refuses(over, status):
    f = 0x30000
    p = O.PolicyArgs(f, f, f, f, 0.2, 0.2, 0.1, 1.0, f, f, f, f, 100)
    for k, v in over.items():
        setattr(p, k, v)
    x = logits_args()
    assert B.lib.z1_policy_loss(ctypes.byref(x), ctypes.byref(p), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(n_rows=-1), B.Z1_EINVAL), (dict(n_pairs=-1), B.Z1_EINVAL), (dict(n_pairs=(1 << 23) + 1), B.Z1_EINVAL),
    (dict(logp=None), B.Z1_EINVAL), (dict(ref_logp=None), B.Z1_EINVAL), (dict(targets=None), B.Z1_EINVAL),
    (dict(cu_seqlens=None), B.Z1_EINVAL), (dict(cu_type=2), B.Z1_EINVAL), (dict(target_type=2), B.Z1_EINVAL),
    (dict(beta=float("inf")), B.Z1_EINVAL), (dict(label_smoothing=1.1), B.Z1_EINVAL), (dict(loss=None), B.Z1_EINVAL),
    (dict(pair_loss=None), B.Z1_EINVAL), (dict(cu_seqlens=0x30004), B.Z1_EALIGN), (dict(dlogp=0x30002), B.Z1_EALIGN),
])
def test_preference_refuses(over, status):
    f = 0x30000
    a = O.PreferenceArgs(10, 2, f, f, f, f, 0, 0, 0.1, 0.0, 1.0, f, f, f, f)
    for k, v in over.items():
        setattr(a, k, v)
    assert B.lib.z1_preference_loss(ctypes.byref(a), None) == status


# ------------------------------------------------------------------ binding

F = torch.float32


def test_binding_refuses_muon_tensors():
    g, m = torch.zeros(4, 6), torch.zeros(4, 6)
    w = torch.zeros(4, 6, dtype=torch.bfloat16)
    ok = dict(shapes=[(4, 6)], grads=[g], momentum=[m], master=[m], weights=[w])
    make = lambda **o: O.z1_muon_create(**{**ok, **o})  # noqa: E731
    with pytest.raises(ValueError, match="current GPU"):
        make()
    with pytest.raises(TypeError, match="weights"):
        make(weights=[m])
    with pytest.raises(TypeError, match="grads"):
        make(grads=[g.half()])
    with pytest.raises(TypeError, match="momentum"):
        make(momentum=[w])
    with pytest.raises(ValueError, match="contiguous"):
        make(grads=[torch.zeros(6, 4).t()])
    with pytest.raises(ValueError, match="elements"):
        make(master=[m[:3]])
    with pytest.raises(ValueError, match="one tensor per matrix"):
        make(grads=[g, g])
    with pytest.raises(ValueError, match="one entry"):
        make(lr_scale=[1.0, 2.0])


def test_binding_refuses_embed_tensors():
    w, ids, out = torch.zeros(5, 4), torch.zeros(3, dtype=torch.long), torch.zeros(3, 4)
    with pytest.raises(ValueError, match="current GPU"):
        O.z1_embed_lookup(w, ids, out)
    with pytest.raises(TypeError, match="ids"):
        O.z1_embed_lookup(w, ids.float(), out)
    with pytest.raises(ValueError, match="ids"):
        O.z1_embed_lookup(w, ids[None], out)
    with pytest.raises(TypeError, match="out: dtype"):
        O.z1_embed_lookup(w, ids, out.half())
    with pytest.raises(ValueError, match="out: shape"):
        O.z1_embed_lookup(w, ids, out[:2])
    with pytest.raises(ValueError, match="not contiguous"):
        O.z1_embed_lookup(torch.zeros(4, 5).t(), ids, out)
    with pytest.raises(ValueError, match="overlap"):
        O.z1_embed_lookup(torch.zeros(4).expand(5, 4), ids, out)
    with pytest.raises(TypeError, match="weight: dtype"):
        O.z1_embed_lookup(w.double(), ids, out)
    ws = torch.zeros(O.z1_embed_grad_workspace(3, 5, 4), dtype=torch.uint8)
    with pytest.raises(ValueError, match="current GPU"):
        O.z1_embed_grad(ids, out, w, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        O.z1_embed_grad(ids, out, w, workspace=ws[:-1])
    with pytest.raises(TypeError, match="dweight"):
        O.z1_embed_grad(ids, out, w.half(), workspace=ws)


def test_binding_refuses_loss_tensors():
    x, y, v = torch.zeros(3, 7), torch.zeros(3, dtype=torch.long), torch.zeros(3)
    with pytest.raises(ValueError, match="current GPU"):
        O.z1_token_logprob(x, y, v, v)
    with pytest.raises(ValueError, match="targets"):
        O.z1_token_logprob(x, y[:2], v, v)
    with pytest.raises(TypeError, match="targets"):
        O.z1_token_logprob(x, y.to(torch.int16), v, v)
    with pytest.raises(ValueError, match="dimensions"):
        O.z1_token_logprob(x[0], y, v, v)
    cu = torch.tensor([0, 1, 3])
    with pytest.raises(ValueError, match="cu_seqlens"):
        O.z1_preference_loss(v, v, y, cu[:2], beta=0.1, loss=v, pair_loss=v)
    with pytest.raises(TypeError, match="logp"):
        O.z1_preference_loss(v.double(), v, y, cu, beta=0.1, loss=v, pair_loss=v)
    with pytest.raises(ValueError, match="ref_logp"):
        O.z1_preference_loss(v, v[:2], y, cu, beta=0.1, loss=v, pair_loss=v)


class Lib:
    """The library's create and destroy without a GPU: each handle is an
    address."""

    def __getattr__(self, name):
        def call(out, *args):
            if name.endswith("create"):
                out._obj.value = 0x1000
            return B.Z1_OK
        return call


def on_host_memory(shape, dtype, alive):
    """A tensor over a numpy array, which `alive` watches."""
    import weakref
    import numpy as np
    a = np.zeros(shape, dtype=np.int32 if dtype == torch.float32 else np.int16)
    alive.append(weakref.ref(a))
    return torch.from_numpy(a).view(dtype)


def test_muon_holds_the_memory_it_is_bound_to(monkeypatch):
    """Not the caller's lists: emptied, or their tensors given other memory
    (as p.data = x does), they leave the handle's addresses valid until close."""
    monkeypatch.setattr(O, "lib", Lib())
    monkeypatch.setattr(O, "_on_gpu", lambda items: None)
    monkeypatch.setattr(O, "_stream", lambda stream: None)
    alive = []
    make = lambda dtype: [on_host_memory((4, 6), dtype, alive), on_host_memory((3, 5), dtype, alive)]  # noqa: E731
    lists = [make(t) for t in (torch.float32, torch.float32, torch.float32, torch.bfloat16, torch.bfloat16)]
    grads, momentum, master, weights, ortho = lists
    m = O.z1_muon_create([(4, 6), (3, 5)], grads, momentum=momentum, master=master, weights=weights, ortho=ortho)
    master[0].data = torch.zeros(4, 6)
    for x in lists:
        x.clear()
    assert all(r() is not None for r in alive) and len(alive) == 10
    m.close()
    assert all(r() is None for r in alive)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), B.Z1_EINVAL), (dict(rows1=0), B.Z1_EINVAL), (dict(ns_steps=0), B.Z1_EINVAL), (dict(reserved=1), B.Z1_EINVAL),
    (dict(master=None), B.Z1_EINVAL), (dict(a=4.0, b=0.0, c=0.0), B.Z1_EINVAL), (dict(at_grad=0), B.Z1_EINVAL),
    (dict(at_weights=0x40001), B.Z1_EALIGN)])
def test_wide_muon_create_refuses_the_same(over, status):
    b, keep = muon_bind(**over)
    h = ctypes.c_void_p(1)
    assert B.lib.z1_muon_create_wide(ctypes.byref(h), ctypes.byref(b), None) == status
    assert h.value is None
    assert B.lib.z1_muon_create_wide(None, ctypes.byref(b), None) == B.Z1_EINVAL
    assert B.lib.z1_muon_create_wide(ctypes.byref(h), None, None) == B.Z1_EINVAL
