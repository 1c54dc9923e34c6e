"""The balance oracle: its gradient against central differences of its losses, and
closed forms."""
import numpy as np
import pytest

from oracle import balance as obal

T, NE, K, ND = 11, 8, 2, 4


def make(seed):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(T, NE))
    return z, np.argsort(-z, axis=1)[:, :K], rng.permutation(NE) % ND


@pytest.mark.parametrize("group_len", [0, 4, 1, 64])
@pytest.mark.parametrize("masked", [False, True])
def test_gradient_is_the_difference_quotient(group_len, masked):
    z, ids, e2v = make(3)
    mask = np.array([1, 1, 0, 1, 0, 0, 0, 0, 1, 1, 1]) if masked else None
    kw = dict(group_len=group_len, mask=mask, coef=0.3, coef_dev=0.2, coef_z=0.1)
    _, counts, grad = obal.loss_and_grad(z, ids, e2v, ND, **kw)
    assert counts.sum() == K * (T if mask is None else mask.sum())
    h = 1e-5
    for i in np.ndindex(T, NE):
        hi, lo = z.copy(), z.copy()
        hi[i] += h
        lo[i] -= h
        num = (obal.loss_and_grad(hi, ids, e2v, ND, **kw)[0][0]
               - obal.loss_and_grad(lo, ids, e2v, ND, **kw)[0][0]) / (2 * h)
        assert abs(grad[i] - num) < 1e-8


def test_closed_forms():
    """Uniform logits: P = 1/Ne, so expert = device = 1 whatever the counts (for devices of
    equal size), and z = log(Ne)^2; everything masked: zero."""
    _, ids, e2v = make(5)
    loss, _, _ = obal.loss_and_grad(np.zeros((T, NE)), ids, e2v, ND, coef=1, coef_dev=1, coef_z=1)
    np.testing.assert_allclose(loss[1:], [1, 1, np.log(NE) ** 2], rtol=1e-12)
    z, ids, e2v = make(6)
    loss, counts, grad = obal.loss_and_grad(z, ids, e2v, ND, mask=np.zeros(T), coef=1, coef_dev=1,
                                            coef_z=1)
    assert not loss.any() and not counts.any() and not grad.any()


def test_all_tokens_on_one_expert():
    """Every token certain of expert 0: f_0 P_0 = Ne / k."""
    z = np.full((T, NE), -60.0)
    z[:, 0] = 60.0
    ids = np.zeros((T, 1), dtype=int)
    loss, counts, _ = obal.loss_and_grad(z, ids, np.arange(NE) % ND, ND, coef=1)
    assert counts[0, 0] == T and loss[1] == pytest.approx(NE)
