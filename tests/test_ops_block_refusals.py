"""Host-side refusals of the norms on both sides of a block and of the low-rank
adapters: an invalid call returns its status before any CUDA work (pointers here are
never followed), and the binding refuses what does not fit before it allocates."""
import ctypes
import os

import pytest
import torch

from mixture_experts_ffn_fp32_gb300 import build as B
from tests.test_ops_devices import On, Stream

pytestmark = pytest.mark.skipif(not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="CUDA toolkit (nvcc) not available")
P = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def A():
    B.build()
    from mixture_experts_ffn_fp32_gb300 import api
    return api


@pytest.fixture(autouse=True)
def nothing_launched(A):
    n = A.launch_count()
    yield
    assert A.launch_count() == n


NORM = dict(R=4, d=8, dtype=0, kind=0, post=1, gate=1, alpha=1.0, eps=1e-5)


def test_block_norm(A):
    def call(x=P, xs=8, y=P, ys=8, g=P, gs=8, pw=P, pb=P, w=P, b=P, out=P, n=P, st=P, **kw):
        c = A.BlockNormConfig(**{**NORM, **kw})
        return A.lib().moe_block_norm(ctypes.byref(c), x, xs, y, ys, g, gs, pw, pb, w, b, out, n, st, None)

    rms = dict(kind=1, pb=None, b=None)
    for kw in (dict(R=-1), dict(d=0), dict(dtype=3), dict(kind=2), dict(post=2), dict(gate=3), dict(gate=-1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(alpha=float("nan")), dict(x=None), dict(xs=7), dict(ys=7),
               dict(x=P + 2), dict(y=P + 1), dict(y=None), dict(g=None), dict(gate=0), dict(g=P + 2),
               dict(gate=2, gs=7), dict(gate=2, g=P + 2), dict(post=0), dict(pw=P + 1), dict(pb=P + 2), dict(w=P + 1),
               dict(b=P + 3), dict(out=None), dict(out=P + 2), dict(n=None), dict(n=P + 1), dict(st=P + 2),
               dict(kind=1), {**rms, "pb": P}, {**rms, "b": P}, dict(y=None, post=0, pw=None, pb=None, gate=0, g=None),
               dict(y=None, post=0, pw=None, pb=None, gate=0, g=None, out=None, n=None, w=None, b=None)):
        assert call(**kw) == A.MOE_ERR_INVALID_ARG, kw
    assert call(d=(1 << 24) + 1, xs=1 << 25, ys=1 << 25) == A.MOE_ERR_UNSUPPORTED
    assert call(R=0, x=None, y=None) == A.MOE_OK  # nothing to do, nothing launched
    assert A.lib().moe_block_norm(None, P, 8, P, 8, P, 8, P, P, P, P, P, P, P, None) == A.MOE_ERR_INVALID_ARG


def test_block_norm_backward(A):
    def call(x=P, xs=8, y=P, ys=8, g=P, gs=8, pw=P, pb=P, w=P, st=P, dn=P, dns=8, dxo=P, dxs=8, dx=P, dy=P, dg=P, dpw=P,
             dpb=P, dw=P, db=P, ws=P, nb=1 << 20, **kw):
        c = A.BlockNormConfig(**{**NORM, **kw})
        return A.lib().moe_block_norm_backward(ctypes.byref(c), x, xs, y, ys, g, gs, pw, pb, w, st, dn, dns, dxo, dxs,
                                               dx, dy, dg, dpw, dpb, dw, db, ws, nb, None)

    for kw in (dict(R=-1), dict(d=0), dict(kind=5), dict(x=None), dict(xs=5), dict(y=None), dict(g=None),
               dict(st=None), dict(st=P + 2), dict(dn=None), dict(dn=None, w=None, dw=None), dict(dns=5), dict(dxs=5),
               dict(dn=P + 2), dict(dxo=P + 1), dict(dn=None, dxo=None, w=None, dw=None, db=None), dict(dx=None),
               dict(dx=P + 2), dict(dy=None), dict(dy=P + 2), dict(dg=P + 2), dict(dpw=P + 2), dict(dpb=P + 1),
               dict(dw=P + 2), dict(db=P + 2), dict(ws=None), dict(ws=P + 4), dict(post=0), dict(kind=1),
               dict(gate=0, g=None), dict(gate=2, dg=P + 2), dict(gate=2, gs=3)):
        assert call(**kw) == A.MOE_ERR_INVALID_ARG, kw
    assert call(nb=8) == A.MOE_ERR_WORKSPACE
    n = ctypes.c_size_t()
    f = A.lib().moe_block_norm_backward_workspace_size
    assert f(None, ctypes.byref(n)) == f(ctypes.byref(A.BlockNormConfig(**NORM)), None) == A.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(A.BlockNormConfig(**{**NORM, "R": -4})), ctypes.byref(n)) == A.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(A.BlockNormConfig(**{**NORM, "R": 0})), ctypes.byref(n)) == A.MOE_OK and n.value == 0


def test_adapter_add(A):
    base = dict(T=8, d=64, N=32, r=16, E=2, dtype=1, out_dtype=1)

    def call(x=P, xs=64, a=P, b=P, sc=P, off=P, rows=P, bs=2 * P, bst=32, out=P, ost=32, ws=P, n=1 << 30, **kw):
        c = A.AdapterConfig(**{**base, **kw})
        return A.lib().moe_adapter_add(ctypes.byref(c), x, xs, a, b, sc, off, rows, bs, bst, out, ost, ws, n, None)

    for kw in (dict(T=-1), dict(d=0), dict(N=0), dict(r=0), dict(E=0), dict(dtype=4), dict(out_dtype=2),
               dict(dtype=0, out_dtype=1), dict(x=None), dict(a=None), dict(b=None), dict(off=None), dict(out=None),
               dict(xs=63), dict(bst=31), dict(ost=31), dict(x=P + 1), dict(a=P + 1), dict(b=P + 1), dict(sc=P + 2),
               dict(off=P + 2), dict(rows=P + 1), dict(bs=P + 1), dict(out=P + 1), dict(ws=None), dict(ws=P + 16),
               dict(bs=P, ost=40)):
        assert call(**kw) == A.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(r=257), dict(E=1025), dict(d=(1 << 24) + 1, xs=1 << 25), dict(N=(1 << 24) + 1), dict(T=(1 << 24) + 1)):
        assert call(**kw) == A.MOE_ERR_UNSUPPORTED, kw
    assert call(n=256) == A.MOE_ERR_WORKSPACE
    assert call(T=0, x=None, out=None) == A.MOE_OK
    n = ctypes.c_size_t()
    f = A.lib().moe_adapter_add_workspace_size
    assert f(None, ctypes.byref(n)) == f(ctypes.byref(A.AdapterConfig(**base)), None) == A.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(A.AdapterConfig(**{**base, "T": 0})), ctypes.byref(n)) == A.MOE_OK and n.value == 0


F, H, I, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture
def here(A, monkeypatch):
    monkeypatch.setattr(A, "_current_device", lambda: 0)

    def refuse(*a, **k):
        raise AssertionError("allocated before the check")
    monkeypatch.setattr(A, "_empty", refuse)


def calls(A):
    def fwd(x, y, w, b, pw, pb, g, **k):
        return A.block_norm(x, y, w, b, pw, pb, g, kind="layer", **k)

    def bwd(x, st, y, dn, dx, w, pw, pb, g, ws, **k):
        return A.block_norm_backward(x, st, y, dn, dx, w, pw, pb, g, kind="layer", ws=ws, **k)

    def add(base, x, a, b, o, r, s, out, ws, **k):
        return A.adapter_add(base, x, a, b, o, r, s, out, ws, **k)
    rows, col = (H, 4, 8), (F, 8)
    return {"block_norm": ([rows, rows, col, col, col, col, rows], fwd),
            "block_norm, a gate per channel": ([rows, rows, col, col, col, col, col], fwd),
            "block_norm_backward": ([rows, (F, 4, 4), rows, rows, rows, col, col, col, rows, (U8, 999)], bwd),
            "adapter_add": ([(F, 4, 6), rows, (H, 3, 2, 8), (H, 3, 6, 2), (I, 4), (I, 4), (F, 3), (F, 4, 6), (U8, 9999)], add)}


NAMES = ["block_norm", "block_norm, a gate per channel", "block_norm_backward", "adapter_add"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_elsewhere_are_refused(A, here, name):
    specs, call = calls(A)[name]
    with pytest.raises(ValueError, match="cuda:0"):
        call(*(On(1, *s) for s in specs))
    for at in range(len(specs)):
        with pytest.raises(ValueError, match="cuda:0"):
            call(*(On(1 if i == at else 0, *s) for i, s in enumerate(specs)))
        with pytest.raises(ValueError):
            call(*(On(-1 if i == at else 0, *s) for i, s in enumerate(specs)))
    with pytest.raises(ValueError, match="cuda:1"):
        call(*(On(0, *s) for s in specs), stream=Stream(1))


@pytest.mark.parametrize("name", NAMES)
def test_types_and_shapes_are_refused(A, here, name):
    specs, call = calls(A)[name]
    for at, (dt, *shape) in enumerate(specs):
        wrong = [(torch.int64, *shape)]
        if dt != U8:
            wrong.append((dt, *shape[:-1], shape[-1] + 1))
        for w in wrong:
            if dt == U8:
                continue  # a workspace is bytes of any type's size: the library checks its length
            if name == "adapter_add" and at == 1 and w[0] == dt:
                continue  # x's width is what a's is checked against
            with pytest.raises(ValueError):
                call(*(On(0, *(w if i == at else s)) for i, s in enumerate(specs)))


def test_arguments_that_do_not_fit(A, here):
    x, v = On(0, H, 4, 8), On(0, F, 8)
    for call in (lambda: A.block_norm(None), lambda: A.block_norm(torch.zeros(4, 8)), lambda: A.block_norm(x, norm=False),
                 lambda: A.block_norm(x, gate=v), lambda: A.block_norm(x, x, kind="group"),
                 lambda: A.block_norm(x, x, bias=v), lambda: A.block_norm(x, x, post_bias=v),
                 lambda: A.block_norm(x, x, post_weight=v, post=False), lambda: A.block_norm(x, post_weight=v),
                 lambda: A.block_norm(x, x, weight=v, norm=False), lambda: A.block_norm(x, On(0, F, 4, 8)),
                 lambda: A.block_norm_backward(x, On(0, F, 2, 4), x),
                 lambda: A.block_norm_backward(x, On(0, F, 4, 4), x, x), lambda: A.block_norm_backward(x, None, x, x),
                 lambda: A.block_norm_backward(x, On(0, F, 2, 4), x, None, x, weight=v),
                 lambda: A.adapter_add(On(0, torch.float16, 4, 6), x, On(0, H, 3, 2, 8), On(0, H, 3, 6, 2), On(0, I, 4)),
                 lambda: A.adapter_add(None, x, On(0, H, 2, 8), On(0, H, 3, 6, 2), On(0, I, 4)),
                 lambda: A.adapter_add(None, x, On(0, H, 3, 2, 8), On(0, H, 3, 6, 4), On(0, I, 4)),
                 lambda: A.alloc_adapter_workspace(4, 8, 8, 2, 1, torch.int8)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: A.block_norm(x, x), lambda: A.block_norm(x)):  # these fit
        with pytest.raises(AssertionError, match="allocated"):
            call()
