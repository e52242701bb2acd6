"""Host-side refusals of the operators around the layer: an invalid call
returns its status before any CUDA work (pointers here are never followed)."""
import ctypes
import os

import pytest
import torch

from mixture_experts_ffn_fp32_gb300 import build as B

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


def test_layer_norm(A):
    f = A.lib().moe_layer_norm

    def call(R=4, d=8, dt=0, x=P, xs=8, g=P, b=P, eps=1e-5, y=P, ys=8, m=P, r=P):
        return f(R, d, dt, x, xs, g, b, eps, y, ys, m, r, None)

    for kw in (dict(R=-1), dict(d=0), dict(dt=3), dict(dt=-1), dict(xs=7), dict(ys=7), dict(xs=-8), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=None), dict(y=None), dict(x=P + 2), dict(y=P + 1), dict(dt=1, x=P + 1),
               dict(g=P + 2), dict(m=P + 3)):
        assert call(**kw) == A.MOE_ERR_INVALID_ARG, kw
    assert call(d=(1 << 24) + 1, xs=1 << 25, ys=1 << 25) == A.MOE_ERR_UNSUPPORTED
    assert call(R=0, x=None, y=None) == A.MOE_OK  # nothing to do, nothing launched


def test_layer_norm_backward(A):
    f = A.lib().moe_layer_norm_backward

    def call(R=4, d=8, dt=0, dy=P, dys=8, x=P, xs=8, m=P, r=P, g=P, dx=P, dxs=8, dg=P, db=P, ws=P, n=1 << 20):
        return f(R, d, dt, dy, dys, x, xs, m, r, g, dx, dxs, dg, db, ws, n, None)

    for kw in (dict(R=-1), dict(d=0), dict(dt=7), dict(dys=5), dict(dxs=5), dict(xs=5), dict(dy=None), dict(x=None),
               dict(m=None), dict(r=None), dict(dx=None), dict(dx=P + 2), dict(ws=None), dict(ws=P + 4), dict(dg=P + 1)):
        assert call(**kw) == A.MOE_ERR_INVALID_ARG, kw
    assert call(n=8) == A.MOE_ERR_WORKSPACE
    n = ctypes.c_size_t()
    assert A.lib().moe_layer_norm_backward_workspace_size(4, 8, None) == A.MOE_ERR_INVALID_ARG
    assert A.lib().moe_layer_norm_backward_workspace_size(-4, 8, ctypes.byref(n)) == A.MOE_ERR_INVALID_ARG


def test_group_route(A):
    L = A.lib()
    base = dict(T=4, E=16, K=2, n_groups=4, topk_groups=2, group_rank=2, score=0, renormalize=1, scale=1.0, dtype=0)

    def call(cfg=None, lg=P, st=16, b=None, i=P, w=P, **kw):
        c = A.GroupRouteConfig(**{**base, **kw})
        fwd = L.moe_group_route(ctypes.byref(c), lg, st, b, i, w, None)
        if b is not None:  # the backward takes no bias
            return {fwd}
        return {fwd, L.moe_group_route_backward(ctypes.byref(c), lg, st, i, w, P, None)}

    for kw in (dict(T=-1), dict(E=0), dict(K=0), dict(K=17), dict(K=9), dict(n_groups=3), dict(n_groups=0),
               dict(topk_groups=0), dict(topk_groups=5), dict(group_rank=0), dict(group_rank=3), dict(score=2),
               dict(renormalize=2), dict(scale=float("nan")), dict(dtype=3), dict(st=15), dict(lg=None), dict(i=None),
               dict(w=None), dict(lg=P + 2), dict(i=P + 1), dict(w=P + 2), dict(b=P + 1)):
        assert call(**kw) == {A.MOE_ERR_INVALID_ARG}, kw
    assert call(E=512, st=512) == {A.MOE_ERR_UNSUPPORTED}
    assert call(E=64, K=17, n_groups=1, topk_groups=1, st=64) == {A.MOE_ERR_UNSUPPORTED}
    assert call(E=256, K=2, n_groups=64, st=256) == {A.MOE_ERR_UNSUPPORTED}
    assert call(T=0, lg=None, i=None, w=None) == {A.MOE_OK}
    assert L.moe_group_route(None, P, 16, None, P, P, None) == A.MOE_ERR_INVALID_ARG


def test_quantize_rows(A):
    f = A.lib().moe_quantize_rows
    ok = [4, 8, 0, P, 8, P, P, None]
    for at, v in ((0, -1), (1, 0), (2, 5), (3, None), (3, P + 2), (4, 7), (5, None), (6, None), (6, P + 2)):
        bad = list(ok)
        bad[at] = v
        assert f(*bad) == A.MOE_ERR_INVALID_ARG, (at, v)
    assert f(0, 8, 0, None, 8, None, None, None) == A.MOE_OK


def test_matmul_int8(A):
    L = A.lib()
    base = dict(M=8, Ma=8, K=64, N=32, E=2, swiglu=0, out_dtype=1)

    def call(a=P, st=64, sa=P, b=P, sb=P, off=P, rows=None, out=P, ws=P, n=1 << 40, **kw):
        c = A.Int8Config(**{**base, **kw})
        return L.moe_matmul_int8(ctypes.byref(c), a, st, sa, b, sb, off, rows, out, ws, n, None)

    for kw in (dict(M=-1), dict(Ma=-1), dict(K=0), dict(N=0), dict(E=0), dict(swiglu=2), dict(swiglu=1, N=33),
               dict(out_dtype=3), dict(off=None), dict(Ma=7), dict(Ma=0, rows=P), dict(a=None), dict(sa=None),
               dict(b=None), dict(sb=None), dict(out=None), dict(st=48), dict(st=72), dict(a=P + 8), dict(b=P + 8),
               dict(out=P + 8), dict(off=P + 2), dict(rows=P + 1), dict(ws=P + 16), dict(ws=None)):
        assert call(**kw) == A.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(K=72, st=80), dict(E=257), dict(K=1 << 18, st=1 << 18)):
        assert call(**kw) == A.MOE_ERR_UNSUPPORTED, kw
    assert call(n=256) == A.MOE_ERR_WORKSPACE
    assert call(M=0, a=None, out=None) == A.MOE_OK
    n = ctypes.c_size_t()
    assert L.moe_matmul_int8_workspace_size(ctypes.byref(A.Int8Config(**{**base, "K": 40})), ctypes.byref(n)) == \
        A.MOE_ERR_UNSUPPORTED
    assert L.moe_matmul_int8_workspace_size(None, ctypes.byref(n)) == A.MOE_ERR_INVALID_ARG


def test_f16_is_no_layer_type(A):
    cfg = A.LayerSpec(T=64, d=64, d_ff=128, E=8, K=2).config()
    cfg.dtype = A.MOE_F16
    n = ctypes.c_size_t()
    assert A.lib().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == A.MOE_ERR_INVALID_ARG


def test_binding_checks(A):
    """The Python binding refuses host tensors, wrong types, shapes and strides."""
    h = torch.zeros(4, 8)
    for call in (lambda: A.layer_norm(h), lambda: A.group_route(h, 2), lambda: A.quantize_rows(h),
                 lambda: A.matmul_int8(h, h, h, h), lambda: A.layer_norm(None),
                 lambda: A.layer_norm_backward(h, h, h, h), lambda: A.group_route_backward(h, h, h)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        A._int8_config(1, 1, 16, 1, 1, False, "int8")
