"""Pins of the logits operators' oracle: scipy's log-softmax and entropy, hand-worked rows, and the gradient
against differences of the loss."""
import numpy as np
import pytest
from scipy.special import log_softmax, logsumexp
from scipy.stats import entropy, rankdata

import oracle.distill as odist
import oracle.logprobs as olp


@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
def test_logprobs_against_scipy(T):
    r = np.random.default_rng(0)
    x = r.standard_normal((6, 97)) * 3
    x[2, 5:60] = -np.inf
    tok = r.integers(0, 5, 6)
    o = olp.logprobs_batch(x, tok, None, 7, T)
    lp = log_softmax(x / T, 1)
    i = np.arange(6)
    assert np.allclose(o["logprob"], lp[i, tok], rtol=1e-13)
    assert np.allclose(o["lse"], logsumexp(x / T, 1), rtol=1e-13)
    assert np.allclose(o["entropy"], entropy(np.exp(lp), axis=1), rtol=1e-12)
    assert (o["rank"] == rankdata(-x, axis=1, method="ordinal")[i, tok]).all()
    assert (o["top_token"] == np.argsort(-x, 1, kind="stable")[:, :7]).all()
    assert np.allclose(o["top_logprob"], np.take_along_axis(lp, o["top_token"], 1), rtol=1e-13)


def test_logprobs_by_hand():
    """Equal logits by index; what is masked is not listed; idle entries."""
    x = np.array([[1.0, 2.0, 2.0, -np.inf], [0.0, 0.0, 0.0, 0.0], [-np.inf] * 4, [np.nan, 1.0, 0.0, 0.0]])
    o = olp.logprobs_batch(x, np.array([2, 3, 1, 0, -1]), np.array([0, 1, 2, 3, 0]), 4, 1.0)
    assert o["top_token"].tolist() == [[1, 2, 0, -1], [0, 1, 2, 3], [-1] * 4, [1, 2, 3, -1], [-1] * 4]
    assert o["rank"].tolist() == [2, 4, 2, 0, 0]
    assert np.isclose(o["entropy"][1], np.log(4)) and o["entropy"][2] == 0 and o["lse"][2] == -np.inf
    assert np.isnan(o["logprob"][3]) and o["logprob"][4] == 0


@pytest.mark.parametrize("mode", [odist.RENORM, odist.REST])
@pytest.mark.parametrize("T", [0.7, 2.0])
def test_distill_gradient_against_differences(mode, T):
    r = np.random.default_rng(1)
    V, K = 23, 6
    z = r.standard_normal(V) * 2
    token = r.choice(V, K, replace=False)
    token[4] = -1
    token[5] = token[0]                            # listed twice
    value = np.log(r.dirichlet(np.ones(K + 1))[:K])
    loss, grad, stats = odist.row_distill(z, token, value, T, mode, 1.5)
    h = 1e-5
    for v in range(V):
        d = np.zeros(V)
        d[v] = h
        up, down = (odist.row_distill(z + s * d, token, value, T, mode, 1.5)[0] for s in (1, -1))
        assert abs((up - down) / (2 * h) - grad[v]) < 1e-8     # second-order term h^2 |f'''| / 6 < 1e-9
    assert np.isclose(stats[0] / T + np.log(stats[1]), logsumexp(z / T)) and abs(grad.sum()) < 1e-13
    seen = np.setdiff1d(np.arange(V), token)
    assert np.isclose(odist.log_rest(stats, T), logsumexp(z[seen] / T) - logsumexp(z / T))


def test_distill_is_a_divergence():
    """0 where the drafter gives the target's probabilities, with the others' share at its place; a full list is
    the plain divergence."""
    r = np.random.default_rng(2)
    z = r.standard_normal(40)
    lp = log_softmax(z)
    top = np.argsort(-lp)[:8]
    assert abs(odist.row_distill(z, top, lp[top], 1.0, odist.REST)[0]) < 1e-14
    assert np.abs(odist.row_distill(z, top, lp[top], 1.0, odist.REST)[1]).max() < 1e-14
    t = log_softmax(r.standard_normal(40))
    want = np.sum(np.exp(t) * (t - lp))
    every = np.arange(40)
    for mode in (odist.RENORM, odist.REST):
        assert np.isclose(odist.row_distill(z, every, t, 1.0, mode)[0], want, rtol=1e-10)


def test_distill_edges():
    z = np.array([1.0, -np.inf, 0.0, 2.0])
    none = np.array([-1, -1])
    for mode in (odist.RENORM, odist.REST):
        loss, grad, stats = odist.row_distill(z, none, np.zeros(2), 1.0, mode)
        assert loss == 0 and not grad.any() and odist.log_rest(stats, 1.0) == 0
    loss, grad, _ = odist.row_distill(z, np.array([1, 3]), np.log([0.5, 0.5]), 1.0, odist.RENORM)
    assert loss == np.inf and grad[1] == -0.5
    assert odist.row_distill(np.full(3, -np.inf), np.array([0]), np.zeros(1), 1.0, odist.RENORM)[0] == np.inf
    assert odist.row_distill(np.full(3, np.nan), np.array([0]), np.zeros(1), 1.0, odist.RENORM, 0.0)[0] == 0
