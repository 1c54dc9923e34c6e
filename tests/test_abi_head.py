"""Host-side refusals of the scored router's entry points: bad options, missing and
misaligned buffers, all before anything launches (a call that got past its checks here,
without a GPU, would report a CUDA error)."""
import ctypes

import pytest
import torch

import synth

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
V = ctypes.c_void_p(256)       # an address that is only compared with NULL and aligned
ODD = ctypes.c_void_p(256 + 2)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def occ():
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    return occ


def desc(occ, **kw):
    return occ.desc_for(synth.CONFIGS["olmoe_fwd"]).replace(**kw)


def route(occ, ds=None, opt=None, **kw):
    a = dict(logits=V, bias=NULL, e2v=V, ids=V, gates=V, vmask=V)
    a.update(kw)
    ds, opt = ds or desc(occ), opt or occ.occult_score_t()
    return occ.lib().occult_route_scored(ctypes.byref(ds), ctypes.byref(opt), *a.values(), NULL)


def route_grad(occ, ds=None, opt=None, **kw):
    a = dict(logits=V, ids=V, dgates=V, dlogits=V)
    a.update(kw)
    ds, opt = ds or desc(occ), opt or occ.occult_score_t()
    return occ.lib().occult_route_scored_grad(ctypes.byref(ds), ctypes.byref(opt), *a.values(), NULL)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [
    dict(score=2), dict(score=-1), dict(n_groups=0), dict(n_groups=7), dict(n_groups=64),
    dict(n_groups=8, keep_groups=0), dict(n_groups=8, keep_groups=9),
    dict(n_groups=16, keep_groups=1),          # four experts cannot hold eight slots
    dict(group_best=0), dict(group_best=3), dict(group_kind=2),
    dict(n_groups=4, keep_groups=2, group_kind=1),   # groups by device: as many as devices
    dict(scale=NAN), dict(scale=INF), dict(bias_rate=NAN), dict(bias_rate=-INF)])
def test_route_scored_refuses_bad_options(occ, kw):
    opt = occ.occult_score_t(**kw)
    assert route(occ, opt=opt) == INVALID
    assert route_grad(occ, opt=opt) == INVALID
    ds = desc(occ)
    assert occ.lib().occult_route_bias_step(ctypes.byref(ds), ctypes.byref(opt), V, 1, V, NULL) == INVALID


def test_route_scored_refuses_other_modes_and_bad_layers(occ):
    for mode in (occ.ROUTE_DEVICE_LIMITED, occ.ROUTE_SCORE_PRUNED, occ.ROUTE_SIMILARITY_PRUNED):
        assert route(occ, ds=desc(occ, route_mode=mode, limit_devices=2)) == INVALID
    assert route(occ, ds=desc(occ, n_vdev=7)) == INVALID
    assert route(occ, ds=desc(occ, n_experts=512)) == UNSUPPORTED
    assert route_grad(occ, ds=desc(occ, T=-1)) == INVALID


@pytest.mark.parametrize("kw", [dict(logits=NULL), dict(e2v=NULL), dict(ids=NULL), dict(gates=NULL),
                                dict(vmask=NULL), dict(logits=ODD), dict(bias=ODD), dict(ids=ODD),
                                dict(gates=ODD), dict(vmask=ODD), dict(e2v=ODD)])
def test_route_scored_refuses_bad_buffers(occ, kw):
    assert route(occ, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(logits=NULL), dict(ids=NULL), dict(dgates=NULL),
                                dict(dlogits=NULL), dict(logits=ODD), dict(dlogits=ODD)])
def test_route_scored_grad_refuses_bad_buffers(occ, kw):
    assert route_grad(occ, **kw) == INVALID


def test_bias_step_refuses(occ):
    ds, opt = desc(occ), occ.occult_score_t()
    f = lambda *a: occ.lib().occult_route_bias_step(ctypes.byref(ds), ctypes.byref(opt), *a, NULL)  # noqa: E731
    assert f(V, 0, V) == INVALID and f(NULL, 1, V) == INVALID and f(V, 1, NULL) == INVALID
    assert f(ODD, 1, V) == INVALID and f(V, 1, ODD) == INVALID


def test_binding_refuses_wrong_tensors(occ):
    ds, opt = desc(occ, T=4), occ.occult_score_t()
    t = torch.zeros(4 * 64)
    with pytest.raises(ValueError, match="CUDA"):
        occ.occult_route_scored(ds, opt, t, t.int(), t.int(), t, t.int())
    with pytest.raises(ValueError, match="required"):
        occ.occult_route_scored(ds, opt, None, t.int(), t.int(), t, t.int())
    with pytest.raises(ValueError, match="required"):
        occ.occult_route_scored_grad(ds, opt, t, None, t, t)
