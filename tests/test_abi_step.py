"""Host-side refusals of the block norm, balance and AdamW entry points: bad options,
missing or misaligned buffers and small workspaces, all before anything launches (a
call that got past its checks here, without a GPU, would report a CUDA error)."""
import ctypes

import pytest
import torch

import synth

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
V = ctypes.c_void_p(256)       # an address that is only compared with NULL and aligned
ODD = ctypes.c_void_p(256 + 2)
NULL = ctypes.c_void_p(0)
BIG = 1 << 40


@pytest.fixture(scope="module")
def occ():
    from combine_top_route_gb300 import build
    build.build()
    import combine_top_route_gb300 as occ
    occ.lib()
    return occ


def desc(occ, **kw):
    return occ.desc_for(synth.CONFIGS["olmoe_fwd"]).replace(**kw)


def norm(occ, ds=None, opt=None, **kw):
    a = dict(r=V, y=V, w_post=V, gate=NULL, w_pre=V, r_out=V, x=V, rstd_post=V, rstd_pre=V)
    a.update(kw)
    ds, opt = ds or desc(occ), opt or occ.occult_norm_t(1e-6, 1.0, 0, occ.OCCULT_BF16)
    return occ.lib().occult_block_norm(ctypes.byref(ds), ctypes.byref(opt), *a.values(), NULL)


@pytest.mark.parametrize("opt", [(0.0, 1.0, 0, 1), (-1e-6, 1.0, 0, 1), (float("nan"), 1.0, 0, 1),
                                 (float("inf"), 1.0, 0, 1), (1e-6, float("nan"), 0, 1),
                                 (1e-6, 1.0, 3, 1), (1e-6, 1.0, -1, 1), (1e-6, 1.0, 0, 2),
                                 (1e-6, 1.0, 1, 1)])      # the last: a gate kind without a gate
def test_block_norm_refuses_bad_options(occ, opt):
    assert norm(occ, opt=occ.occult_norm_t(*opt)) == INVALID


@pytest.mark.parametrize("kw", [
    dict(r=NULL), dict(r_out=NULL), dict(x=NULL), dict(gate=V),
    dict(w_post=NULL), dict(w_pre=NULL),                 # a row factor without its norm
    dict(y=NULL), dict(y=NULL, w_post=NULL, rstd_post=NULL),   # r_out without y
    dict(y=NULL, w_post=NULL, rstd_post=NULL, r_out=NULL, w_pre=NULL, x=NULL, rstd_pre=NULL),
    dict(w_pre=NULL, rstd_pre=NULL),                     # x without w_pre
    dict(r=ODD), dict(y=ODD), dict(x=ODD), dict(r_out=ODD), dict(w_pre=ODD), dict(w_post=ODD)])
def test_block_norm_refuses_bad_buffers(occ, kw):
    assert norm(occ, **kw) == INVALID


def test_block_norm_refuses_wide_rows_and_bad_layers(occ):
    assert norm(occ, ds=desc(occ, d=16448)) == UNSUPPORTED
    assert norm(occ, ds=desc(occ, d=2050)) == UNSUPPORTED
    assert norm(occ, ds=desc(occ, n_vdev=7)) == INVALID


def norm_bwd(occ, ds=None, opt=None, ws_bytes=BIG, **kw):
    a = dict(dr_out=V, dx=V, r_out=V, y=V, w_post=V, gate=V, w_pre=V, rstd_post=V, rstd_pre=V,
             dr=V, dy=V, dw_post=V, dgate=V, dw_pre=V, ws=V)
    a.update(kw)
    ds, opt = ds or desc(occ), opt or occ.occult_norm_t(1e-6, 1.0, 1, occ.OCCULT_BF16)
    return occ.lib().occult_block_norm_bwd(ctypes.byref(ds), ctypes.byref(opt), *a.values(),
                                           ctypes.c_size_t(ws_bytes), NULL)


@pytest.mark.parametrize("kw", [
    dict(dr=NULL), dict(dy=NULL), dict(dx=NULL), dict(r_out=NULL), dict(dw_pre=NULL),
    dict(dw_post=NULL), dict(dgate=NULL), dict(gate=NULL), dict(rstd_pre=NULL),
    dict(rstd_post=NULL), dict(w_post=NULL), dict(w_pre=NULL),
    dict(y=NULL), dict(dr_out=NULL, w_pre=NULL, dw_pre=NULL, dx=NULL),   # no gradient arrives
    dict(dr_out=ODD), dict(dx=ODD), dict(dr=ODD), dict(dy=ODD), dict(ws=ODD)])
def test_block_norm_bwd_refuses_bad_buffers(occ, kw):
    assert norm_bwd(occ, **kw) == INVALID


def test_block_norm_bwd_refuses_a_small_workspace(occ):
    need = occ.workspace_size(desc(occ), occ.WS_BLOCK_NORM_BWD)
    assert need > 0
    assert norm_bwd(occ, ws_bytes=need - 1) == WORKSPACE
    assert norm_bwd(occ, ws=NULL) == WORKSPACE


def balance(occ, ds=None, opt=None, ws_bytes=BIG, **kw):
    a = dict(logits=V, ids=V, e2v=V, mask=NULL, counts=V, grad_w=V, loss=V, ws=V)
    a.update(kw)
    ds, opt = ds or desc(occ), opt or occ.occult_balance_t(0.01, 0.0, 0.0, 0)
    return occ.lib().occult_balance_loss(ctypes.byref(ds), ctypes.byref(opt), *a.values(),
                                         ctypes.c_size_t(ws_bytes), NULL)


@pytest.mark.parametrize("kw", [dict(logits=NULL), dict(ids=NULL), dict(e2v=NULL),
                                dict(counts=NULL), dict(grad_w=NULL), dict(loss=NULL),
                                dict(logits=ODD), dict(ids=ODD), dict(ws=ODD)])
def test_balance_loss_refuses_bad_buffers(occ, kw):
    assert balance(occ, **kw) == INVALID


def test_balance_refuses_bad_options_and_workspaces(occ):
    assert balance(occ, opt=occ.occult_balance_t(0.01, 0, 0, -1)) == INVALID
    ds, opt = desc(occ), occ.occult_balance_t(0.01, 0, 0, 100)
    need = occ.balance_workspace_size(ds, opt)
    assert balance(occ, opt=opt, ws_bytes=need - 1) == WORKSPACE
    assert balance(occ, opt=opt, ws=NULL) == WORKSPACE
    L, g = occ.lib(), occ.lib().occult_balance_grad
    assert L.occult_balance_workspace_size(ctypes.byref(ds), NULL, V) == INVALID
    assert L.occult_balance_workspace_size(ctypes.byref(ds), ctypes.byref(opt), NULL) == INVALID
    d, o = ctypes.byref(ds), ctypes.byref(opt)
    assert g(d, o, NULL, V, NULL, NULL, V, 0, NULL) == INVALID
    assert g(d, o, V, NULL, NULL, NULL, V, 0, NULL) == INVALID
    assert g(d, o, V, V, NULL, NULL, NULL, 0, NULL) == INVALID
    assert g(d, o, V, V, NULL, NULL, V, 2, NULL) == INVALID
    assert g(d, o, ODD, V, NULL, NULL, V, 0, NULL) == INVALID
    assert g(d, NULL, V, V, NULL, NULL, V, 0, NULL) == INVALID


def adamw(occ, opt=None, n=1, **kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1, state_bits=32)
    o = occ.occult_adamw_t(**{**base, **(opt or {})})
    a = dict(param=256, master=None, grad=256, m=256, v=256, m_exp=256, v_exp=256, n=100, first=0,
             dtype=occ.OCCULT_BF16)
    a.update(kw)
    return occ.lib().occult_adamw(ctypes.byref(o), ctypes.byref(occ.occult_param_t(**a)), n, NULL)


@pytest.mark.parametrize("opt", [dict(step=0), dict(state_bits=16), dict(beta1=1.0),
                                 dict(beta2=1.0), dict(beta1=-0.1), dict(beta2=float("nan")),
                                 dict(eps=0.0), dict(eps=float("nan")), dict(lr=float("nan")),
                                 dict(lr=float("inf")), dict(weight_decay=float("nan")),
                                 dict(reserved=1)])
def test_adamw_refuses_bad_options(occ, opt):
    assert adamw(occ, opt) == INVALID


@pytest.mark.parametrize("kw", [dict(param=None), dict(grad=None), dict(m=None), dict(v=None),
                                dict(n=-1), dict(first=-1), dict(dtype=2), dict(reserved=1),
                                dict(dtype=0, master=256), dict(param=258), dict(grad=260),
                                dict(master=264), dict(m=257), dict(v=258)])
def test_adamw_refuses_bad_tensors(occ, kw):
    assert adamw(occ, **kw) == INVALID


def test_adamw_refuses_missing_exponents_and_tables(occ):
    assert adamw(occ, dict(state_bits=8), m_exp=None) == INVALID
    assert adamw(occ, dict(state_bits=8), v_exp=None) == INVALID
    assert adamw(occ, n=-1) == INVALID
    assert occ.lib().occult_adamw(NULL, V, 1, NULL) == INVALID
    r = occ.lib().occult_adamw_read
    assert r(V, V, ctypes.c_int64(-1), 0, V, NULL) == INVALID
    assert r(V, V, ctypes.c_int64(4), 2, V, NULL) == INVALID
    assert r(NULL, V, ctypes.c_int64(4), 0, V, NULL) == INVALID
    assert r(ODD, V, ctypes.c_int64(4), 0, V, NULL) == INVALID


def test_binding_refuses_what_the_records_cannot_say(occ):
    """CPU tensors, mixed state types and masters of fp32 parameters."""
    f = torch.zeros(8)
    with pytest.raises(ValueError):
        occ.adamw_table([dict(param=f, grad=f, m=f, v=f)])            # not on a GPU
    with pytest.raises(ValueError):
        occ.adamw_table([dict(param=f, grad=f, m=f, v=f),
                         dict(param=f, grad=f, m=f.to(torch.uint8), v=f)])
    with pytest.raises(ValueError):
        occ.adamw_table([dict(param=f, master=f, grad=f, m=f, v=f)])
    table = occ.adamw_table([])
    with pytest.raises(ValueError):
        occ.occult_adamw(occ.occult_adamw_t(state_bits=8, step=1), table)


def test_packed_record_is_the_struct(occ):
    """The binding packs occult_param_t as bytes: the same size and field offsets."""
    rec = occ.occult_param_t()
    vals = [0x1000 * (i + 1) for i in range(7)] + [12345678901, 98765432109, 1, 0]
    assert occ._RECORD.size == ctypes.sizeof(rec)
    occ._RECORD.pack_into(rec, 0, *vals)
    got = [getattr(rec, n) for n, _ in rec._fields_]
    assert got == vals


@pytest.mark.parametrize("kw", [dict(lr=float("inf")), dict(lr=float("nan"))])
def test_a_refused_step_is_not_counted(occ, kw):
    """The step's number (of the bias corrections and the draws) and the rate stay."""
    opt = occ.OccultAdamW([], [], lr=1e-3)
    opt.opt.step = 7
    with pytest.raises(occ.OccultError):
        opt.step(stream=0, **kw)
    assert opt.opt.step == 7 and opt.opt.lr == 1e-3 and opt.opt.grad_scale is None


def test_balance_grad_refuses_weights_off_a_word(occ):
    """They need no whole 16 bytes, but a float must be where a float can be."""
    ds, opt = desc(occ), occ.occult_balance_t(0.01, 0.0, 0.0, 0)
    g = occ.lib().occult_balance_grad
    args = lambda w: (ctypes.byref(ds), ctypes.byref(opt), V, w, NULL, NULL, V, 0, NULL)  # noqa: E731
    assert g(*args(ODD)) == INVALID


def test_words_off_a_word_are_refused(occ):
    """Buffers that are read and written by single words: at an odd address a kernel would
    fault, so the call says so."""
    for k in ("rstd_post", "rstd_pre"):
        assert norm(occ, **{k: ODD}) == INVALID
        assert norm_bwd(occ, **{k: ODD}) == INVALID
    for k in ("dw_post", "dgate", "dw_pre"):
        assert norm_bwd(occ, **{k: ODD}) == INVALID
    for k in ("e2v", "counts", "grad_w", "loss"):
        assert balance(occ, **{k: ODD}) == INVALID
    ds, opt = desc(occ), occ.occult_balance_t(0.01, 0.0, 0.0, 0)
    assert occ.lib().occult_balance_grad(ctypes.byref(ds), ctypes.byref(opt), V, V, NULL, ODD, V, 0,
                                         NULL) == INVALID
    assert adamw(occ, dict(grad_scale=258)) == INVALID
