"""The head's oracle: its gradients against central differences, and closed forms."""
import numpy as np
import pytest

from oracle import head

T, D, V, K = 7, 5, 11, 4


def make(seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    ids[2, 1:] = -1          # a short row
    ids[4, 0] = V            # no teacher
    labels = rng.integers(0, V, T)
    labels[1] = -100
    labels[4] = V            # row 4 counts nowhere
    tl = rng.normal(size=(T, K)) * 2
    tl[5, 2] = -np.inf
    return rng.normal(size=(T, D)), rng.normal(size=(V, D)), labels, ids, tl


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("teacher", [True, False])
def test_gradients_are_the_difference_quotients(tau, teacher):
    x, w, labels, ids, tl = make(1)
    kw = dict(labels=labels, tau=tau, coef=0.7, coef_z=0.01, dloss=1.0)
    if teacher:
        kw.update(t_ids=ids, t_logits=tl, coef_kd=0.4)
    out = head.losses(x, w, **kw)
    h = 1e-5
    for name, a in (("dx", x), ("dw", w)):
        for i in np.ndindex(*a.shape):
            keep = a[i]
            a[i] = keep + h
            hi = head.losses(x, w, grads=False, **kw)["loss"][0]
            a[i] = keep - h
            lo = head.losses(x, w, grads=False, **kw)["loss"][0]
            a[i] = keep
            assert abs(out[name][i] - (hi - lo) / (2 * h)) < 1e-8, (name, i)
    assert (out["dx"][4] == 0).all() and out["lse"][4] == 0 and out["token_loss"][1] == 0


def test_closed_forms():
    """Zero logits: ce = log V, z = log(V)^2; a teacher equal to the student over the whole
    vocabulary: kd = 0 at any temperature, and no gradient."""
    labels = np.arange(T)
    out = head.losses(np.zeros((T, D)), np.ones((V, D)), labels)
    np.testing.assert_allclose(out["loss"][[1, 3]], [np.log(V), np.log(V) ** 2], rtol=1e-12)
    x, w, _, _, _ = make(2)
    ids = np.tile(np.arange(V), (T, 1))
    out = head.losses(x, w, t_ids=ids, t_logits=x @ w.T, tau=3.0, coef=0.0, coef_kd=1.0)
    assert abs(out["loss"][2]) < 1e-12 and np.abs(out["dx"]).max() < 1e-12


def test_a_teacher_without_a_finite_logit_adds_nothing():
    x, w, _, ids, _ = make(3)
    out = head.losses(x, w, t_ids=ids, t_logits=np.full((T, K), -np.inf), coef=0.0, coef_kd=1.0)
    assert out["loss"][2] == 0 and (out["dx"] == 0).all() and (out["dw"] == 0).all()
