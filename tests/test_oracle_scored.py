"""The scored router's oracle: its gradient against central differences of its gates,
hand-made choices, and the bias step."""
import numpy as np
import pytest

from oracle import scored


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_is_the_difference_quotient(sigmoid, renorm):
    rng = np.random.default_rng(4)
    z, dg = rng.normal(size=(6, 8)), rng.normal(size=(6, 3))
    z[0, 2] = -np.inf
    e2v = np.arange(8) % 4
    kw = dict(sigmoid=sigmoid, scale=2.5, renorm=renorm)
    ids, _, _ = scored.route(z, 3, e2v, n_groups=4, keep=2, best=2, **kw)
    got = scored.grad(z, ids, dg, **kw)

    def total(zz):
        out = 0.0
        for t in range(len(zz)):
            s, _ = scored.scores(zz[t], sigmoid)
            g = s[ids[t]]
            out += 2.5 * (dg[t] * (g / g.sum() if renorm else g)).sum()
        return out

    h = 1e-6
    for i in np.ndindex(*z.shape):
        if np.isinf(z[i]):
            assert got[i] == 0
            continue
        hi, lo = z.copy(), z.copy()
        hi[i] += h
        lo[i] -= h
        assert abs(got[i] - (total(hi) - total(lo)) / (2 * h)) < 1e-8


def test_choices():
    e2v = np.array([0, 1, 0, 1, 2, 2])
    z = np.array([[0.0, 1.0, 1.0, -1.0, 3.0, -np.inf]])
    # by logit, ties to the lower expert
    assert scored.route(z, 4, e2v)[0].tolist() == [[4, 1, 2, 0]]
    # a bias reorders, the gates stay scores
    ids, g, vm = scored.route(z, 2, e2v, bias=np.array([1.0, 0, 0, 0.5, -1, 0]), renorm=False)
    assert ids.tolist() == [[0, 3]] and vm.tolist() == [0b11]
    np.testing.assert_allclose(g, [[0.5, 1 / (1 + np.e)]])
    # two blocks of three; the second one's best two are 3 and -1: sigmoid sum 1.22 < 1.46
    assert scored.route(z, 2, e2v, n_groups=2, keep=1, best=2)[0].tolist() == [[1, 2]]
    assert scored.route(z, 2, e2v, n_groups=2, keep=1, best=1)[0].tolist() == [[4, 3]]
    # by devices {0, 2}, {1, 3}, {4, 5}: of the last only one expert is on
    assert scored.route(z, 2, e2v, n_groups=3, keep=1, best=1, by_vdev=True)[0].tolist() == [[4, 5]]
    # everything off: the lowest experts of the lowest groups, gates 0
    ids, g, _ = scored.route(np.full((1, 6), -np.inf), 2, e2v, n_groups=3, keep=1, sigmoid=False)
    assert ids.tolist() == [[0, 1]] and (g == 0).all()


def test_bias_step():
    b = scored.bias_step(np.zeros(4), [[3, 1, 0, 4], [1, 1, 0, 6]], 0.1)
    np.testing.assert_allclose(b, [0.0, 0.1, 0.1, -0.1])


@pytest.mark.parametrize("best", [1, 2])
def test_worths_of_any_size(best):
    """Groups are kept by their worth however small it is, and true ties fall to the lower one."""
    e2v = np.zeros(6, int)
    kw = dict(n_groups=3, keep=2, best=best)
    z = np.array([[0.0, -1, -70, -71, -69.5, -71], [0.0, -1, -69.5, -71, -69.5, -71], [-80.0, -90, -90, -81, -79, -90]])
    for sigmoid in (True, False):
        ids = scored.route(z, 4, e2v, sigmoid=sigmoid, **kw)[0]
        assert np.sort(ids, axis=1).tolist() == [[0, 1, 4, 5], [0, 1, 2, 3], [0, 1, 4, 5]]
    # x and -x: 1 for every x
    z = np.array([[3.3, -3.3, 0.0, 0.0, 17.7, -17.7]])
    assert scored.route(z, 4, e2v, n_groups=3, keep=2, best=2)[0].tolist() == [[0, 2, 3, 1]]
    assert scored.route(z, 2, e2v, n_groups=3, keep=1, best=1)[0].tolist() == [[4, 5]]
