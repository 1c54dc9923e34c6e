"""Host-side refusals of the scored router's and the output head's entry points: bad
options, missing and misaligned buffers, small workspaces, all before anything launches (a call that got past its checks here,
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


# ---- the output head ------------------------------------------------------------------
ODD16 = ctypes.c_void_p(256 + 8)   # on a word, off a 16-byte boundary
BIG = 1 << 40


def head(occ, step, ds=None, opt=None, ws_bytes=BIG, **kw):
    a = dict(x=V, w=V, labels=V, t_ids=NULL, t_logits=NULL)
    if step:
        a.update(dloss=NULL)
    a.update(lse=NULL, token_loss=NULL, loss=V)
    if step:
        a.update(dx=V, dw=V)
    a.update(ws=V)
    a.update({k: v for k, v in kw.items() if k in a})
    ds, opt = ds or desc(occ), opt or occ.occult_head_t(vocab=1000)
    f = occ.lib().occult_head_step if step else occ.lib().occult_head_loss
    return f(ctypes.byref(ds), ctypes.byref(opt), *a.values(), ws_bytes, NULL)


@pytest.mark.parametrize("kw", [
    dict(vocab=0), dict(vocab=-5), dict(topk=-1), dict(piece=-1), dict(grad_dtype=2), dict(coef=-1.0),
    dict(coef=NAN), dict(coef_kd=INF), dict(coef_z=NAN), dict(coef_kd=-0.5),
    dict(topk=4, temperature=0.0), dict(topk=4, temperature=NAN), dict(topk=4, temperature=0.2),
    dict(topk=4, temperature=11.0)])
def test_head_refuses_bad_options(occ, kw):
    opt = occ.occult_head_t(**{"vocab": 1000, **kw})
    more = dict(t_ids=V, t_logits=V) if kw.get("topk", 0) > 0 else {}
    assert head(occ, True, opt=opt, **more) == INVALID
    assert head(occ, False, opt=opt, **more) == INVALID
    n = ctypes.c_size_t(0)
    assert occ.lib().occult_head_workspace_size(ctypes.byref(desc(occ)), ctypes.byref(opt), 1,
                                                ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("kw", [
    dict(x=NULL), dict(w=NULL), dict(loss=NULL), dict(labels=NULL),          # neither labels nor a teacher
    dict(t_ids=V, t_logits=V), dict(t_ids=V),                                # a teacher with topk 0
    dict(labels=NULL, token_loss=V), dict(x=ODD16), dict(w=ODD16), dict(ws=ODD16), dict(labels=ODD),
    dict(loss=ODD), dict(lse=ODD), dict(token_loss=ODD)])
def test_head_refuses_bad_buffers(occ, step, kw):
    assert head(occ, step, **kw) == INVALID


def test_head_refuses_bad_teachers_and_gradients(occ):
    opt = occ.occult_head_t(vocab=1000, topk=8)
    assert head(occ, True, opt=opt) == INVALID                      # no teacher given
    assert head(occ, True, opt=opt, t_ids=V) == INVALID
    assert head(occ, True, opt=opt, t_ids=ODD, t_logits=V) == INVALID
    assert head(occ, False, opt=opt, labels=NULL, token_loss=V, t_ids=V, t_logits=V) == INVALID
    assert head(occ, True, dx=NULL, dw=NULL) == INVALID
    assert head(occ, True, dx=ODD16) == INVALID and head(occ, True, dw=ODD16) == INVALID
    assert head(occ, True, dloss=ODD) == INVALID


def test_head_refuses_what_it_does_not_run(occ):
    assert head(occ, True, opt=occ.occult_head_t(vocab=1000, topk=129), t_ids=V, t_logits=V) == UNSUPPORTED
    assert head(occ, True, opt=occ.occult_head_t(vocab=1 << 29)) == UNSUPPORTED
    assert head(occ, True, ds=desc(occ, d=16448)) == UNSUPPORTED
    assert head(occ, False, ds=desc(occ, d=2050)) == UNSUPPORTED
    few = dict(n_experts=1, top_k=1, n_vdev=1)
    assert head(occ, False, ds=desc(occ, T=(1 << 30) + 1, **few)) == UNSUPPORTED
    assert head(occ, False, ds=desc(occ, T=1 << 24, **few), opt=occ.occult_head_t(vocab=1 << 17)) == UNSUPPORTED
    assert head(occ, True, ds=desc(occ, T=1 << 25, n_experts=8, top_k=2),
                opt=occ.occult_head_t(vocab=1000, topk=100), t_ids=V, t_logits=V) == UNSUPPORTED


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("T,V_,K,dtype", [(1, 1, 0, 1), (4096, 50304, 64, 1), (32768, 151936, 0, 1),
                                          (257, 1009, 5, 0)])
def test_head_workspace(occ, step, T, V_, K, dtype):
    """The size asked for is the size refused below; a step's logits stay within 1 GiB."""
    ds, opt = desc(occ, T=T, dtype=dtype), occ.occult_head_t(vocab=V_, topk=K)
    need = occ.head_workspace_size(ds, opt, step=step)
    more = dict(t_ids=V, t_logits=V) if K else {}
    assert head(occ, step, ds=ds, opt=opt, ws_bytes=need - 1, **more) == WORKSPACE
    assert head(occ, step, ds=ds, opt=opt, ws=NULL, **more) == WORKSPACE
    if T == 32768:
        rest = 2 * T * 2048 + 4 * T * 40 + 12 * 4096 * 1200   # x's copy, rows, sums
        assert need < (1 << 30) + rest + 4 * 64 * 4096 * 2048
    n = ctypes.c_size_t(0)
    bad = lambda *a: occ.lib().occult_head_workspace_size(ctypes.byref(ds), ctypes.byref(opt), *a)  # noqa: E731
    assert bad(2, ctypes.byref(n)) == INVALID and bad(1, NULL) == INVALID


def test_head_binding_refuses_wrong_tensors(occ):
    ds, opt = desc(occ, T=4), occ.occult_head_t(vocab=10)
    t = torch.zeros(4 * 2048, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        occ.occult_head_loss(ds, opt, t, t, torch.zeros(4), torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="required"):
        occ.occult_head_step(ds, opt, t, None, torch.zeros(4), torch.zeros(8, dtype=torch.uint8))
