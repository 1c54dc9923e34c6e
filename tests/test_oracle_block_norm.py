"""The block norm oracle: its gradients against central differences of its forward,
and closed forms."""
import numpy as np
import pytest

from oracle import block_norm as onorm

EPS = 1e-3
T, D = 3, 8


def make(post, pre, gate, rng):
    g = {"none": None, "channel": rng.normal(size=D), "token": rng.normal(size=(T, 1))}[gate]
    return dict(r=rng.normal(size=(T, D)), y=rng.normal(size=(T, D)),
                w_post=rng.normal(size=D) if post else None, gate=g,
                w_pre=rng.normal(size=D) if pre else None)


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_backward_is_the_difference_quotient(post, pre, gate):
    rng = np.random.default_rng(7)
    v = make(post, pre, gate, rng)
    a = 0.7
    up_r, up_x = rng.normal(size=(T, D)), rng.normal(size=(T, D))

    def f(**kw):
        o = onorm.forward(eps=EPS, res_scale=a, **{**v, **kw})
        return (o["r_out"] * up_r).sum() + ((o["x"] * up_x).sum() if pre else 0.0)

    fw = onorm.forward(eps=EPS, res_scale=a, **v)
    got = onorm.backward(up_r, up_x if pre else None, fw["r_out"], v["y"], v["w_post"], v["gate"],
                         v["w_pre"], fw.get("rstd_post"), fw.get("rstd_pre"), a)
    name = {"r": "dr", "y": "dy", "w_post": "dw_post", "gate": "dgate", "w_pre": "dw_pre"}
    h = 1e-5
    for key, val in v.items():
        if val is None:
            assert name[key] not in got
            continue
        num = np.zeros(val.shape)
        for i in np.ndindex(*val.shape):
            hi, lo = val.copy(), val.copy()
            hi[i] += h
            lo[i] -= h
            num[i] = (f(**{key: hi}) - f(**{key: lo})) / (2 * h)
        # truncation h^2 f''' and cancellation 1e-16 |f| / h: both below 1e-8 here
        np.testing.assert_allclose(got[name[key]].reshape(val.shape), num, rtol=0, atol=1e-7)


def test_norm_before_the_first_block_only():
    rng = np.random.default_rng(1)
    r, w, up = rng.normal(size=(T, D)), rng.normal(size=D), rng.normal(size=(T, D))
    fw = onorm.forward(r, w_pre=w, eps=EPS)
    assert set(fw) == {"x", "rstd_pre"}
    got = onorm.backward(None, up, r, w_pre=w, rstd_pre=fw["rstd_pre"])
    h = 1e-5
    for i in np.ndindex(T, D):
        hi, lo = r.copy(), r.copy()
        hi[i] += h
        lo[i] -= h
        num = ((onorm.forward(hi, w_pre=w, eps=EPS)["x"] - onorm.forward(lo, w_pre=w, eps=EPS)["x"])
               * up).sum() / (2 * h)
        assert abs(got["dr"][i] - num) < 1e-7


def test_closed_forms():
    """A row of equal values c > 0 normalises to w (eps -> 0); a zero row to zeros."""
    w = np.arange(1.0, 9.0)
    fw = onorm.forward(np.full((1, D), 5.0), w_pre=w, eps=1e-30)
    np.testing.assert_allclose(fw["x"][0], w, rtol=1e-12)
    fw = onorm.forward(np.zeros((1, D)), w_pre=w, eps=1e-6)
    assert (fw["x"] == 0).all() and fw["rstd_pre"][0] == pytest.approx(1e3)
