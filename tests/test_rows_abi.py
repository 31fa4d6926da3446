"""Refusals of the row operators' entry points on the host (no GPU needed): bad arguments return
before anything is launched. The pointers are fake addresses that are never dereferenced."""

import ctypes

import pytest
import torch

import mhc_hyper_connection_02_b200 as mhc

A = 1 << 40
INV, ALIAS, SMALL = mhc.MHC_ERR_INVALID_ARG, mhc.MHC_ERR_ALIAS, mhc.MHC_ERR_WORKSPACE_TOO_SMALL


def at(i):
    return A + (i << 34)


@pytest.fixture(scope="module")
def L():
    from mhc_hyper_connection_02_b200 import build
    build.build()
    return mhc.lib()


def f32(v):
    return ctypes.c_float(v)


def norm(L, **o):
    a = dict(x=at(0), xs=64, dt=0, g=at(1), b=at(2), wd=2, y=at(3), m=at(4), r=at(5), T=8, H=64,
             eps=1e-6)
    a.update(o)
    return L.mhc_layer_norm(a["x"], a["xs"], a["dt"], a["g"], a["b"], a["wd"], a["y"], a["m"],
                            a["r"], a["T"], a["H"], f32(a["eps"]), None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), mhc.MHC_OK), (dict(T=-1), INV), (dict(H=0), INV), (dict(xs=63), INV),
    (dict(dt=3), INV), (dict(wd=1), INV), (dict(wd=3), INV), (dict(eps=0.0), INV),
    (dict(eps=float("nan")), INV), (dict(x=None), INV), (dict(y=None), INV),
    (dict(x=at(0) + 1), INV), (dict(g=at(1) + 2), INV), (dict(m=at(4) + 2), INV),
    (dict(H=1 << 29, xs=1 << 29), INV), (dict(T=1 << 31), INV), (dict(xs=1 << 41), INV),
    (dict(y=at(0) + 2), ALIAS), (dict(y=at(0), xs=65), ALIAS), (dict(m=at(5)), ALIAS),
    (dict(m=at(0)), ALIAS), (dict(g=at(3)), ALIAS), (dict(r=at(3) + 64), ALIAS)])
def test_layer_norm_refusals(L, bad, status):
    assert norm(L, **bad) == status


def norm_bwd(L, **o):
    a = dict(dy=at(0), ds=64, x=at(1), xs=64, dt=0, g=at(2), wd=2, m=at(3), r=at(4), dx=at(5),
             dg=at(6), db=at(7), ws=at(8), T=8, H=64)
    a.update(o)
    need = mhc.layer_norm_backward_workspace_bytes(a["T"], a["H"])
    n = o.get("wsb", need)
    return L.mhc_layer_norm_backward(a["dy"], a["ds"], a["x"], a["xs"], a["dt"], a["g"], a["wd"],
                                     a["m"], a["r"], a["dx"], a["dg"], a["db"], a["ws"], n, a["T"],
                                     a["H"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0, dg=None, db=None), mhc.MHC_OK), (dict(T=-1), INV), (dict(H=0), INV),
    (dict(ds=63), INV), (dict(xs=63), INV), (dict(dt=-1), INV), (dict(wd=1), INV),
    (dict(dy=None), INV), (dict(m=None), INV), (dict(dx=None), INV), (dict(dg=at(6) + 1), INV),
    (dict(dx=at(5) + 1), INV), (dict(ws=None), SMALL), (dict(wsb=16), SMALL),
    (dict(ws=at(8) + 16), INV), (dict(dx=at(0)), ALIAS), (dict(dx=at(1)), ALIAS),
    (dict(dg=at(7)), ALIAS), (dict(dg=at(2)), ALIAS), (dict(ws=at(5)), ALIAS),
    (dict(db=at(8)), ALIAS)])
def test_layer_norm_backward_refusals(L, bad, status):
    assert norm_bwd(L, **bad) == status


def test_layer_norm_backward_workspace(L):
    f = mhc.layer_norm_backward_workspace_bytes
    assert f(0, 64) == 0 and f(8, 0) == 0 and f(-1, 64) == 0
    for T, H in ((1, 1), (1, 7168), (8192, 7168), (5, 16391)):
        assert f(T, H) > 0 and f(T, H) % 256 == 0


def lp(L, **o):
    a = dict(z=at(0), zs=640, dt=0, y=at(1), tau=1.0, lp=at(2), e=at(3), top=4, ti=at(4), tl=at(5),
             st=at(6), T=8, V=640)
    a.update(o)
    return L.mhc_token_logprobs(a["z"], a["zs"], a["dt"], a["y"], f32(a["tau"]), a["lp"], a["e"],
                                a["top"], a["ti"], a["tl"], a["st"], a["T"], a["V"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), mhc.MHC_OK), (dict(T=-1), INV), (dict(V=0), INV), (dict(zs=639), INV),
    (dict(dt=9), INV), (dict(tau=0.0), INV), (dict(tau=-1.0), INV), (dict(tau=float("inf")), INV),
    (dict(tau=float("nan")), INV), (dict(tau=1e-44), INV), (dict(top=33), INV), (dict(top=-1), INV),
    (dict(top=5, V=4), INV), (dict(z=None), INV), (dict(y=None), INV), (dict(lp=None), INV),
    (dict(ti=None), INV), (dict(tl=None), INV),
    (dict(y=None, lp=None, e=None, top=0, st=None), INV),
    (dict(z=at(0) + 1), INV), (dict(y=at(1) + 4), INV), (dict(st=at(6) + 4), INV),
    (dict(ti=at(4) + 4), INV), (dict(T=1 << 29), INV), (dict(V=1 << 29, zs=1 << 29), INV),
    (dict(lp=at(0)), ALIAS), (dict(e=at(2)), ALIAS), (dict(st=at(1)), ALIAS),
    (dict(ti=at(5)), ALIAS), (dict(tl=at(0) + 64), ALIAS)])
def test_token_logprobs_refusals(L, bad, status):
    assert lp(L, **bad) == status


def lpb(L, **o):
    a = dict(z=at(0), zs=640, dt=0, y=at(1), tau=1.0, st=at(2), g=at(3), h=at(4), e=at(5), d=at(6),
             ds=640, T=8, V=640)
    a.update(o)
    return L.mhc_token_logprobs_backward(a["z"], a["zs"], a["dt"], a["y"], f32(a["tau"]), a["st"],
                                         a["g"], a["h"], a["e"], a["d"], a["ds"], a["T"], a["V"],
                                         None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), mhc.MHC_OK), (dict(T=-1), INV), (dict(V=0), INV), (dict(zs=1), INV),
    (dict(ds=639), INV), (dict(dt=3), INV), (dict(tau=0.0), INV), (dict(z=None), INV),
    (dict(st=None), INV), (dict(d=None), INV), (dict(g=None, h=None), INV), (dict(y=None), INV),
    (dict(e=None), INV), (dict(st=at(2) + 4), INV), (dict(d=at(6) + 1), INV),
    (dict(d=at(0) + 2), ALIAS), (dict(d=at(0), ds=641), ALIAS), (dict(d=at(3)), ALIAS),
    (dict(d=at(2) - 16), ALIAS), (dict(d=at(1)), ALIAS)])
def test_token_logprobs_backward_refusals(L, bad, status):
    assert lpb(L, **bad) == status


def kd(L, **o):
    a = dict(z=at(0), zs=640, dt=0, i=at(1), t=at(2), td=2, tau=1.0, l=at(3), w=at(4), st=at(5),
             T=8, V=640, K=16)
    a.update(o)
    return L.mhc_distill_topk(a["z"], a["zs"], a["dt"], a["i"], a["t"], a["td"], f32(a["tau"]),
                              a["l"], a["w"], a["st"], a["T"], a["V"], a["K"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), mhc.MHC_OK), (dict(T=-1), INV), (dict(V=0), INV), (dict(K=0), INV),
    (dict(K=1025), INV), (dict(td=4), INV), (dict(dt=4), INV), (dict(tau=0.0), INV),
    (dict(zs=2), INV), (dict(i=None), INV), (dict(t=None), INV), (dict(l=None), INV),
    (dict(w=None), INV), (dict(st=None), INV), (dict(i=at(1) + 4), INV), (dict(t=at(2) + 2), INV),
    (dict(w=at(2)), ALIAS), (dict(l=at(0)), ALIAS), (dict(st=at(4)), ALIAS), (dict(T=1 << 29), INV)])
def test_distill_refusals(L, bad, status):
    assert kd(L, **bad) == status


def kdb(L, **o):
    a = dict(z=at(0), zs=640, dt=0, i=at(1), w=at(2), st=at(3), g=at(4), tau=1.0, d=at(5), ds=640,
             T=8, V=640, K=16)
    a.update(o)
    return L.mhc_distill_topk_backward(a["z"], a["zs"], a["dt"], a["i"], a["w"], a["st"], a["g"],
                                       f32(a["tau"]), a["d"], a["ds"], a["T"], a["V"], a["K"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), mhc.MHC_OK), (dict(T=-1), INV), (dict(V=-4), INV), (dict(K=0), INV),
    (dict(K=1025), INV), (dict(tau=-2.0), INV), (dict(ds=4), INV), (dict(i=None), INV),
    (dict(w=None), INV), (dict(st=None), INV), (dict(g=None), INV), (dict(d=None), INV),
    (dict(d=at(0) + 2), ALIAS), (dict(d=at(2)), ALIAS), (dict(d=at(1)), ALIAS)])
def test_distill_backward_refusals(L, bad, status):
    assert kdb(L, **bad) == status


def test_bindings_refuse_what_is_not_a_cuda_row_tensor(L):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        mhc.layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        mhc.token_logprobs(x)
    with pytest.raises(ValueError, match="bfloat16"):
        mhc.token_logprobs(x.double())
    with pytest.raises(ValueError, match="bfloat16"):
        mhc.distill_topk(x.to(torch.int32), None, None)
    with pytest.raises(TypeError):
        mhc.layer_norm([1.0])
