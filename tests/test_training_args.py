"""Host checks of the norm's and the router's training entry points: bad
arguments come back as documented before anything is enqueued (no GPU
needed), workspace sizes, and the binding's refusal of CPU tensors."""

import ctypes
import math
import os

import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call fails its checks first
OK, INVAL, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from mixture_experts_layer_04_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_04_amd import build
        build.build()
    return _lib.lib()


def test_rms_norm(L):
    def call(x=FAKE, res=FAKE, rf=0, w=FAKE, wf=0, T=4, H=256, eps=1e-6, q=0, h=FAKE, y=FAKE, qo=None, s=None):
        return L.moe_rms_norm(x, res, rf, w, wf, T, H, eps, q, h, y, qo, s, None)
    assert call(T=0) == OK
    assert call(T=-1) == INVAL and call(T=(1 << 24) + 1) == INVAL and call(H=0) == INVAL
    assert call(eps=-1e-6) == INVAL and call(eps=math.nan) == INVAL and call(eps=math.inf) == INVAL
    assert call(rf=2) == INVAL and call(wf=-1) == INVAL and call(q=3) == INVAL
    assert call(x=None) == INVAL and call(w=None) == INVAL and call(y=None) == INVAL
    assert call(res=None) == INVAL                      # h without a residual
    assert call(q=1, qo=None, s=FAKE) == INVAL and call(q=2, qo=FAKE, s=None) == INVAL
    assert call(q=1, qo=ctypes.c_void_p(0x1004), s=FAKE) == INVAL  # q is 8-byte aligned
    assert call(H=32769) == UNSUPPORTED
    assert call(q=1, H=192, qo=FAKE, s=FAKE) == UNSUPPORTED and call(q=2, H=48, qo=FAKE, s=FAKE) == UNSUPPORTED


def test_rms_norm_grad(L):
    def call(dy=FAKE, dh=None, h=FAKE, hf=0, w=FAKE, wf=0, T=4, H=256, eps=1e-6, dx=FAKE, dw=FAKE, ws=FAKE,
             n=1 << 30):
        return L.moe_rms_norm_grad(dy, dh, h, hf, w, wf, T, H, eps, dx, dw, ws, n, None)
    assert call(T=-1) == INVAL and call(H=0) == INVAL and call(eps=-1.0) == INVAL and call(hf=2) == INVAL
    assert call(dy=None) == INVAL and call(h=None) == INVAL and call(w=None) == INVAL and call(dx=None) == INVAL
    assert call(ws=None) == INVAL and call(n=16) == WORKSPACE and call(H=40000) == UNSUPPORTED
    assert call(T=0, dw=None, ws=None, n=0) == OK
    assert L.moe_rms_norm_grad_workspace_size(-1, 8) == 0 and L.moe_rms_norm_grad_workspace_size(4, 40000) == 0
    # one fp32 row per row in flight, behind the control block
    assert L.moe_rms_norm_grad_workspace_size(1, 256) >= 65536 + 1024


def test_balance_loss(L):
    def call(lg=FAKE, ids=FAKE, off=None, T=16, E=32, k=4, ns=0, S=1, sc=0, out=FAKE, ws=FAKE, n=1 << 30):
        return L.moe_balance_loss(lg, ids, None, off, T, E, k, ns, S, sc, out, FAKE, FAKE, FAKE, ws, n, None)
    assert call(T=-1) == INVAL and call(E=0) == INVAL and call(E=1025) == INVAL and call(k=0) == INVAL
    assert call(k=33) == INVAL and call(k=17) == INVAL and call(k=16, ns=1) == INVAL and call(ns=2) == INVAL
    assert call(S=0) == INVAL and call(S=2) == INVAL and call(off=FAKE, S=(1 << 20) + 1) == INVAL
    assert call(sc=3) == INVAL and call(lg=None) == INVAL and call(ids=None) == INVAL and call(out=None) == INVAL
    assert call(T=300, ws=None) == INVAL and call(T=300, n=1000) == WORKSPACE
    assert L.moe_balance_loss_workspace_size(256, 256, 1) == 0  # one launch, no scratch memory
    assert L.moe_balance_loss_workspace_size(-1, 8, 1) == 0 and L.moe_balance_loss_workspace_size(8, 8, 0) == 0
    small, large = (L.moe_balance_loss_workspace_size(T, 256, 4) for T in (16, 100000))
    assert 65536 < small < large


def test_route_grad(L):
    def call(lg=FAKE, off=None, T=16, E=32, k=4, ns=0, S=1, sc=0, dw=FAKE, dl=FAKE, c=FAKE, tk=FAKE, out=FAKE):
        return L.moe_route_grad(lg, FAKE, None, off, T, E, k, ns, S, sc, 1, 1.0, dw, dl, c, tk, out, None)
    assert call(T=0) == OK
    assert call(k=0) == INVAL and call(S=3) == INVAL and call(sc=-1) == INVAL and call(lg=None) == INVAL
    assert call(dw=None, dl=None) == INVAL and call(c=None) == INVAL and call(tk=None) == INVAL
    assert call(out=None) == INVAL


def test_gate_grad(L):
    def call(x=FAKE, g=FAKE, gf=1, d=FAKE, di=None, T=16, H=256, E=32, dx=FAKE, dg=FAKE, ws=FAKE, n=1 << 30):
        return L.moe_gate_grad(x, g, gf, d, di, T, H, E, dx, dg, ws, n, None)
    assert call(T=-1) == INVAL and call(H=100) == INVAL and call(H=0) == INVAL and call(E=1025) == INVAL
    assert call(gf=2) == INVAL and call(dx=None, dg=None) == INVAL and call(dx=None, di=FAKE) == INVAL
    assert call(d=None) == INVAL and call(x=None) == INVAL and call(g=None) == INVAL and call(ws=None) == INVAL
    odd = ctypes.c_void_p(0x1008)  # 8-byte aligned only
    assert call(x=odd) == INVAL and call(dx=odd) == INVAL and call(di=odd) == INVAL and call(ws=odd) == INVAL
    assert call(n=70000) == WORKSPACE and call(T=0, dg=None) == OK
    assert L.moe_gate_grad_workspace_size(4, 100, 8) == 0


def test_norm_layer(L):
    def call(x=FAKE, res=FAKE, nw=FAKE, eps=1e-6, T=4, H=256, h=FAKE, ws=FAKE, n=1 << 30, k=2, rf=0):
        return L.moe_norm_layer(x, res, rf, nw, 0, eps, FAKE, 1, None, 0, FAKE, None, FAKE, None, T, H, 8, 128, k, 0, 1,
                                1, 0, 1, 1.0, 16, math.inf, h, FAKE, None, None, ws, n, None)
    assert call(T=0) == OK
    assert call(nw=None) == INVAL and call(res=None) == INVAL and call(eps=-1.0) == INVAL and call(rf=5) == INVAL
    assert call(k=9) == INVAL and call(H=200) == INVAL and call(ws=None) == INVAL
    need = L.moe_norm_layer_workspace_size(4, 256, 8, 128, 2, 0, 16, 0)
    assert need > L.moe_layer_workspace_size(4, 256, 8, 128, 2, 0, 16, 0)
    assert call(n=need - 1) == WORKSPACE


def test_the_binding_refuses_cpu_tensors():
    import mixture_experts_layer_04_amd as moe
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    lg, ids = torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32)
    for f in (lambda: moe.rms_norm(x, torch.ones(128)), lambda: moe.rms_norm_grad(x, x, torch.ones(128)),
              lambda: moe.balance_loss(lg, ids), lambda: moe.route_grad(lg, ids, d_weights=torch.zeros(2, 1)),
              lambda: moe.gate_grad(x, torch.zeros(4, 128), lg),
              lambda: moe.norm_layer(x, torch.ones(128), torch.zeros(4, 128), None, torch.zeros(4, 256, 128),
                                     torch.zeros(4, 128, 128), 1)):
        with pytest.raises(ValueError):
            f()
